// Dense products with bias, activation and residual in their epilogue, and
// their gradients.
#include <math.h>

#include <algorithm>
#include <type_traits>

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
// sigmoid_f (kt_common.hpp) is within a few roundings; a NaN stays one
__device__ __forceinline__ float sigmoid_lin(float u) { return u != u ? u : sigmoid_f(u); }

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case KT_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
    case KT_ACT_SILU: return fmaxf(z, -128.f) * sigmoid_lin(z);  // (the sigmoid is 0 there: -infinity gives -0, not NaN)
    // (erfc keeps the digits of a small Phi, where 1 + erf has none left; -infinity gives -0)
    case KT_ACT_GELU: return 0.5f * fmaxf(z, -16.f) * erfcf(-z * kInvSqrt2);
    case KT_ACT_GELU_TANH: return fmaxf(z, -16.f) * sigmoid_lin(z != z ? z : gelu_tanh_arg(z));
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
      return 0.5f * erfcf(-z * kInvSqrt2) + c * expf(-0.5f * c * c) * kInvSqrt2Pi;
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

// C[m, n] = sum_k A(m, k) B(n, k) with the epilogue of one of the three products:
//   forward      A = x  [T][K]       B = W [N][K]       contraction contiguous in both
//   grad_input   A = dz [T][N]       B = W [N][K]       contraction (N) contiguous in A, across B's rows
//   d_weight     A = dz [T][N]       B = x [T][K]       contraction (T) across both operands' rows
// An operand whose contraction is contiguous lies in memory as [rows][ld], the
// other kind as [contraction][ld].
enum LinearKind { kLinFwd, kLinDx, kLinDw };

constexpr int kMaxPlanes = 3;
constexpr int kDxPlanes = 2;  // for grad_input

struct LinearGemm {
  const uint16_t *a, *b;
  int64_t lda, ldb;      // row pitch (elements, a multiple of 8)
  int64_t a_width;       // columns of A's rows that exist (a multiple of 8), for a contraction across them
  int64_t M, N, K;
  int64_t a_plane;       // elements from one of A's planes to the next, where A is the sum of bf16 planes
  int planes;            // grad_input: how many (1 or kDxPlanes; d_weight's are a constant of the kernel)
  int splits;            // the steps of the contraction are dealt to so many blocks; over 1: part
  float* part;           // [splits][M][pn] partial sums
  int64_t pn;            // N rounded up to a multiple of 8
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

// One output, ACT the forward's activation.
template <int KIND, int ACT>
__device__ __forceinline__ void finish1(const LinearGemm& g, int64_t m, int64_t n, float v) {
  const int64_t i = m * g.N + n;
  if (KIND == kLinDw) {
    float* o = static_cast<float*>(g.out) + i;
    *o = (g.accumulate ? *o : 0.f) + g.scale * v;
    return;
  }
  if (KIND == kLinFwd) {
    if (g.bias) v += g.bias[n];
    if (g.preact) g.preact[i] = float_to_bf16(v);
    v = act_value(ACT, v);
  }
  if (g.residual) v += bf16_to_float(g.residual[i]);
  if (KIND == kLinFwd && g.out_f32)
    static_cast<float*>(g.out)[i] = v;
  else
    static_cast<uint16_t*>(g.out)[i] = float_to_bf16(v);
}

// Outputs m, n .. n + 7 (n a multiple of 8; those below N exist).
template <int KIND, int ACT>
__device__ __forceinline__ void finish8(const LinearGemm& g, int64_t m, int64_t n, float (&v)[8]) {
  const int64_t i = m * g.N + n;
  if ((g.N & 7) == 0) {  // rows of whole, aligned 16-byte pieces
    auto put16 = [&](uint16_t* p) {
      *reinterpret_cast<u32x4*>(p) =
          u32x4{pack2(float_to_bf16(v[0]), float_to_bf16(v[1])), pack2(float_to_bf16(v[2]), float_to_bf16(v[3])),
                pack2(float_to_bf16(v[4]), float_to_bf16(v[5])), pack2(float_to_bf16(v[6]), float_to_bf16(v[7]))};
    };
    auto put32 = [&](float* p) {
      *reinterpret_cast<floatx4*>(p) = floatx4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<floatx4*>(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
    };
    u32x4 res = {};
    if (KIND != kLinDw && g.residual) res = *reinterpret_cast<const u32x4*>(g.residual + i);
    if (KIND == kLinDw) {
      float* o = static_cast<float*>(g.out) + i;
      floatx4 lo = {}, hi = {};
      if (g.accumulate) {
        lo = *reinterpret_cast<const floatx4*>(o);
        hi = *reinterpret_cast<const floatx4*>(o + 4);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = (r < 4 ? lo[r & 3] : hi[r & 3]) + g.scale * v[r];
      put32(o);
      return;
    }
    if (KIND == kLinFwd) {
      if (g.bias) {
        const floatx4 lo = *reinterpret_cast<const floatx4*>(g.bias + n);
        const floatx4 hi = *reinterpret_cast<const floatx4*>(g.bias + n + 4);
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] += r < 4 ? lo[r & 3] : hi[r & 3];
      }
      if (g.preact) put16(g.preact + i);
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = act_value(ACT, v[r]);
    }
    if (g.residual) {
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] += bf16_to_float((uint16_t)(res[r >> 1] >> (16 * (r & 1))));
    }
    if (KIND == kLinFwd && g.out_f32)
      put32(static_cast<float*>(g.out) + i);
    else
      put16(static_cast<uint16_t*>(g.out) + i);
    return;
  }
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (n + r < g.N) finish1<KIND, ACT>(g, m, n + r, v[r]);
}

// body(ACT as a constant) for the forward's activation
template <int KIND, typename F>
__device__ __forceinline__ void with_act(int act, F body) {
  if (KIND != kLinFwd) {
    body(std::integral_constant<int, KT_ACT_NONE>());
    return;
  }
  switch (act) {
    case KT_ACT_RELU: body(std::integral_constant<int, KT_ACT_RELU>()); break;
    case KT_ACT_SILU: body(std::integral_constant<int, KT_ACT_SILU>()); break;
    case KT_ACT_GELU: body(std::integral_constant<int, KT_ACT_GELU>()); break;
    case KT_ACT_GELU_TANH: body(std::integral_constant<int, KT_ACT_GELU_TANH>()); break;
    default: body(std::integral_constant<int, KT_ACT_NONE>());
  }
}

// contraction values per step of the tiles
constexpr int linear_step(int planes) { return planes == 1 ? 64 : 32; }

// 16 zero bytes that copies past the end of a contraction read
__device__ const uint32_t kZero16[4] = {0, 0, 0, 0};

__device__ __forceinline__ uint64_t uniform64(const void* p) {
  const uint64_t v = (uint64_t)p;
  // (readfirstlane gives an int: without the casts the low half's sign would fill the high half)
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  return (uint64_t)hi << 32 | lo;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// dma16 with a wave-uniform base and a 32-bit byte offset per lane.  A load may read a scalar that a
// vector instruction wrote (readfirstlane) after five wait states; the compiler does not see the load.
__device__ __forceinline__ void dma16_off(const void* base, uint32_t off, uint32_t lds_base) {
  const uint32_t lb = __builtin_amdgcn_readfirstlane(lds_base);
  const uint64_t ub = uniform64(base);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(ub), "s"(lb)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// One operand's tile of R rows (or columns) x BK contraction values in LDS, filled by 16-byte copies straight from memory: a wave's copy
// fills 1024 consecutive bytes, so the arrangement is made on the source side.
//
// Contiguous contraction: row r at r * 128, its 16-byte chunk c (8 values) at
// position c ^ (r >> 1 & 7).  A fragment read takes one chunk of 16 consecutive
// rows; even rows lie in the lower and odd rows in the upper 32 banks, eight
// different chunks of each: all 64 banks once.
//
// Contraction across rows: value k of all R columns at k * 2R, the 32-byte pair
// p (16 columns) at position p ^ h(k).  A fragment (16 columns x 8 values per
// lane) is two transposing reads, each of 4 values k for 16 columns per 16
// lanes; h(k) = (k & 3) | (k >> 3 & 1) << 2 spreads the 8 rows that two 16-lane
// groups read together over all banks.
template <int R, bool ACROSS, int BK>
struct LinTile {
  static_assert(ACROSS || BK == 64, "rows of 128 bytes");
  static constexpr int kBytes = R * 2 * BK;
  static constexpr int kCopies = kBytes / 1024;

  // the pair swizzle of contraction value k
  __device__ static int spread(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

  // tile row (contraction value if ACROSS) and element within it that lane l of copy q fills
  __device__ static void place(int q, int l, int& row, int& col) {
    if (ACROSS) {
      const int at = q * 64 + l;  // 16-byte chunk of the tile
      row = at / (R / 8);
      const int pos = at % (R / 8);
      col = (((pos >> 1) ^ spread(row)) * 2 + (pos & 1)) * 8;
    } else {
      row = q * 8 + (l >> 3);
      col = ((l & 7) ^ ((row >> 1) & 7)) * 8;
    }
  }

  // the 8 contraction values ks * 32 + 8 (lane / 16) .. + 7 of row (column) r0 + lane % 16
  __device__ static u32x4 fragment(const uint8_t* tile, int r0, int ks, int lane) {
    const int g = lane >> 4, j = lane & 15;
    if (ACROSS) {
      const int h = spread(8 * g + (j >> 2));
      const uint8_t* p = tile + (ks * 32 + 8 * g + (j >> 2)) * (2 * R) + (((r0 >> 4) ^ h) * 32) + (j & 3) * 8;
      typedef short4_t __attribute__((address_space(3))) * lds_p;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p)));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p + 8 * R)));
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    }
    const int row = r0 + j;
    return *reinterpret_cast<const u32x4*>(tile + row * 128 + (((ks * 4 + g) ^ ((row >> 1) & 7)) * 16));
  }
};

// A block of WM x WN waves computes BM x BN outputs, each wave BM / WM x BN / WN
// of them as 16 x 16 MFMA tiles.  Two LDS buffers: while one step's tiles are
// multiplied, the next step's are copied into the other.  A step is 64
// contraction values, or 32 of PLANES = 3 planes of A, which share B's tile (the
// planes one after another would copy and read B three times: d_weight of 4096 x
// 7168 x 384 from fp32 gradients 84 us so against 77, of 8192 x 7168 x 2048 602
// against 588).
//
// Bound by the MFMAs: at 8192 x 7168 x 2048 they are busy 58% of the time at the
// 2.0 GHz that the chip's power then leaves, the LDS's index unit 23% and without bank
// conflicts; the rest is the turn from one step to the next and the epilogue.
// Reached there: 1.27 PFLOP/s forward and 1.24 in d_weight with three planes (1.21
// with one), where a library's plain product runs at 1.31.  At a contraction of 384 it is
// 0.57 to 0.68: of a tile's six steps nothing covers the first copies and the epilogue.
template <int KIND, int BM, int BN, int WM, int WN, int PLANES>
__global__ __launch_bounds__(64 * WM* WN, WM* WN > 4 ? 1 : 2) void k_linear(LinearGemm g) {
  constexpr bool kAcrossA = KIND == kLinDw, kAcrossB = KIND != kLinFwd;
  constexpr int BK = linear_step(PLANES);
  typedef LinTile<BM, kAcrossA, BK> TA;
  typedef LinTile<BN, kAcrossB, BK> TB;
  constexpr int kWaves = WM * WN, kFm = BM / WM / 16, kFn = BN / WN / 16;
  constexpr int kCa = TA::kCopies / kWaves, kCb = TB::kCopies / kWaves, kOffB = PLANES * TA::kBytes;
  static_assert(PLANES == 1 || (PLANES == kMaxPlanes && KIND == kLinDw), "planes");
  __shared__ __align__(1024) uint8_t lds[2][kOffB + TB::kBytes];

  // tiles: each XCD (blocks reach them in turn) takes a contiguous run of the
  // order below, in which kRows rows of tiles are walked column by column, so
  // that the operand rows a run shares stay in that XCD's L2
  constexpr int kRows = 4;
  const int mt = (int)((g.M + BM - 1) / BM), nt = (int)((g.N + BN - 1) / BN), tiles = mt * nt;
  const int xcd = blockIdx.x & 7, q8 = tiles >> 3, r8 = tiles & 7;
  const int tile = __builtin_amdgcn_readfirstlane(xcd * q8 + min(xcd, r8) + (int)(blockIdx.x >> 3));
  const int span = kRows * nt, grp = tile / span, in = tile - grp * span;
  const int rows = min(kRows, mt - grp * kRows);
  const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(grp * kRows + in % rows) * BM;
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(in / rows) * BN;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the steps of this split
  const int dx_planes = KIND == kLinDx ? g.planes : 1;
  const int total = (int)((g.K + BK - 1) / BK) * dx_planes;
  const int s0 = __builtin_amdgcn_readfirstlane((int)((int64_t)total * blockIdx.y / g.splits));
  const int s1 = __builtin_amdgcn_readfirstlane((int)((int64_t)total * (blockIdx.y + 1) / g.splits));

  // byte offsets of this lane's copies from the tile's first element; rows and
  // columns past the operand's end repeat its last ones (their outputs are not stored)
  uint32_t off_a[kCa], off_b[kCb];
#pragma unroll
  for (int c = 0; c < kCa; ++c) {
    int row, col;
    TA::place(wave * kCa + c, lane, row, col);
    off_a[c] = kAcrossA ? (uint32_t)((row * g.lda + min((int64_t)col, g.a_width - 8 - m0)) * 2)
                        : (uint32_t)((min((int64_t)row, g.M - 1 - m0) * g.lda + col) * 2);
  }
#pragma unroll
  for (int c = 0; c < kCb; ++c) {
    int row, col;
    TB::place(wave * kCb + c, lane, row, col);
    off_b[c] = kAcrossB ? (uint32_t)((row * g.ldb + min((int64_t)col, g.ldb - 8 - n0)) * 2)
                        : (uint32_t)((min((int64_t)row, g.N - 1 - n0) * g.ldb + col) * 2);
  }
  const uint8_t* base_a = reinterpret_cast<const uint8_t*>(g.a + (kAcrossA ? m0 : m0 * g.lda));
  const uint8_t* base_b = reinterpret_cast<const uint8_t*>(g.b + (kAcrossB ? n0 : n0 * g.ldb));
  const int64_t step_a = kAcrossA ? 2 * BK * g.lda : 2 * BK, step_b = kAcrossB ? 2 * BK * g.ldb : 2 * BK;

  // The next copy's step.  Every tile walks the contraction in the same order, so
  // that equal rows of A give equal outputs wherever they stand: a token's logits,
  // and the choice made on them, do not depend on its place in the batch.  (Each XCD
  // starting at another eighth spreads the reads over the memory channels: 16384 x
  // 7168 x 384 in 113 us instead of 116, but with sums in another order per XCD.)
  int ks = s0;
  // grad_input's planes take turns at each piece of the contraction, so that B's tile comes from L2 the second time.
  auto copy = [&](int buf) {
    const bool two = KIND == kLinDx && dx_planes == kDxPlanes;
    const int kc = two ? ks >> 1 : ks, second = two ? ks & 1 : 0;
    const uint8_t* pb = base_b + kc * step_b;
    const uint32_t la = lds_addr(&lds[buf][0]) + wave * kCa * 1024;
    const uint32_t lb = lds_addr(&lds[buf][kOffB]) + wave * kCb * 1024;
    const bool whole = (int64_t)(kc + 1) * BK <= g.K;
    const int left = (int)(g.K - (int64_t)kc * BK);  // values that exist
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
      const uint8_t* pa = base_a + 2 * (p + second) * g.a_plane + kc * step_a;
      if (whole) {
#pragma unroll
        for (int c = 0; c < kCa; ++c) dma16_off(pa, off_a[c], la + p * TA::kBytes + c * 1024);
      } else {
#pragma unroll
        for (int c = 0; c < kCa; ++c) {
          int row, col;
          TA::place(wave * kCa + c, lane, row, col);
          dma16((kAcrossA ? row : col) < left ? (const void*)(pa + off_a[c]) : kZero16, la + p * TA::kBytes + c * 1024);
        }
      }
    }
    if (whole) {
#pragma unroll
      for (int c = 0; c < kCb; ++c) dma16_off(pb, off_b[c], lb + c * 1024);
    } else {
#pragma unroll
      for (int c = 0; c < kCb; ++c) {
        int row, col;
        TB::place(wave * kCb + c, lane, row, col);
        dma16((kAcrossB ? row : col) < left ? (const void*)(pb + off_b[c]) : kZero16, lb + c * 1024);
      }
    }
    ++ks;
  };

  const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
  floatx4 acc[kFm][kFn] = {};
  struct FragsA {
    u32x4 v[kFm];
  };
  struct FragsB {
    u32x4 v[kFn];
  };
  // the fragments of half h of the step in buffer buf
  auto load_a = [&](FragsA& f, int buf, int h) {
#pragma unroll
    for (int i = 0; i < kFm; ++i) f.v[i] = TA::fragment(&lds[buf][0], wm + 16 * i, h, lane);
  };
  auto load_b = [&](FragsB& f, int buf, int h) {
#pragma unroll
    for (int j = 0; j < kFn; ++j) f.v[j] = TB::fragment(&lds[buf][kOffB], wn + 16 * j, h, lane);
  };
  auto multiply = [&](const FragsA& a, const FragsB& b) {
#pragma unroll
    for (int i = 0; i < kFm; ++i)
#pragma unroll
      for (int j = 0; j < kFn; ++j) acc[i][j] = mfma_bf16(b.v[j], a.v[i], acc[i][j]);
  };
  constexpr int kReadsA = kFm * (kAcrossA ? 2 : 1), kReadsB = kFn * (kAcrossB ? 2 : 1);
  // spreads a phase's LDS reads over its MFMAs
  auto spread = [](auto reads, auto products) {
    constexpr int kReads = decltype(reads)::value, kMfma = decltype(products)::value;
    constexpr int kPer = kMfma / kReads > 0 ? kMfma / kReads : 1;
#pragma unroll
    for (int r = 0; r < kReads; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  std::integral_constant<int, kReadsA + kReadsB> reads;
  std::integral_constant<int, kReadsA / 2> reads_half;
  std::integral_constant<int, kReadsA / 2 + kReadsB> reads_half_b;
  std::integral_constant<int, kFm * kFn> products;
  std::integral_constant<int, kFm * kFn / 2> products_half;
  auto fence = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // every wave holds the rest of its tile in registers: the next step's copies, issued a step ago, must have
  // landed, and the copies of the step after it may overwrite this step's buffer
  auto turn_over = [&](int s, int buf) {
    wait_vm_lgkm<0>();
    fence();
    __builtin_amdgcn_s_barrier();
    fence();
    if (s + 2 < s1) copy(buf);
  };
  // A step is two halves of 32 contraction values, or three planes of 32.  While
  // one is multiplied, the next one's fragments are read (the next step's first
  // ones during the last).
  if (s0 < s1) {
    copy(0);
    if (s0 + 1 < s1) {
      copy(1);
      wait_vm_lgkm<PLANES * kCa + kCb>();
    } else {
      wait_vm_lgkm<0>();
    }
    fence();
    __builtin_amdgcn_s_barrier();
    fence();
    FragsB b0, b1;
    load_b(b0, 0, 0);
    if constexpr (PLANES == 1) {
      FragsA a0, a1;
      load_a(a0, 0, 0);
      int buf = 0;
      for (int s = s0; s + 1 < s1; ++s) {
        load_b(b1, buf, 1);
        load_a(a1, buf, 1);
        multiply(a0, b0);
        spread(reads, products);
        fence();
        turn_over(s, buf);
        buf ^= 1;
        load_b(b0, buf, 0);
        load_a(a0, buf, 0);
        multiply(a1, b1);
        spread(reads, products);
      }
      load_b(b1, buf, 1);
      load_a(a1, buf, 1);
      multiply(a0, b0);
      multiply(a1, b1);
    } else {
      // by halves of A's rows: six half planes a step, each read while the one before is multiplied
      constexpr int kHalf = kFm / 2;
      u32x4 x[kHalf], y[kHalf];
      auto load_half = [&](u32x4(&f)[kHalf], int buf, int p, int part) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
          f[i] = TA::fragment(&lds[buf][p * TA::kBytes], wm + 16 * (part * kHalf + i), 0, lane);
      };
      auto multiply_half = [&](const u32x4(&f)[kHalf], auto part) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
          for (int j = 0; j < kFn; ++j) {
            constexpr int first = decltype(part)::value * kHalf;
            acc[first + i][j] = mfma_bf16(b0.v[j], f[i], acc[first + i][j]);
          }
      };
      std::integral_constant<int, 0> lower;
      std::integral_constant<int, 1> upper;
      // everything but the last half plane; y holds that one at the end
      auto five = [&](int buf) __attribute__((always_inline)) {
        load_half(y, buf, 0, 1);
        multiply_half(x, lower);
        spread(reads_half, products_half);
        load_half(x, buf, 1, 0);
        multiply_half(y, upper);
        spread(reads_half, products_half);
        load_half(y, buf, 1, 1);
        multiply_half(x, lower);
        spread(reads_half, products_half);
        load_half(x, buf, 2, 0);
        multiply_half(y, upper);
        spread(reads_half, products_half);
        load_half(y, buf, 2, 1);
        multiply_half(x, lower);
        spread(reads_half, products_half);
      };
      load_half(x, 0, 0, 0);
      int buf = 0;
      for (int s = s0; s + 1 < s1; ++s) {
        five(buf);
        fence();
        turn_over(s, buf);
        buf ^= 1;
        load_b(b1, buf, 0);
        load_half(x, buf, 0, 0);
        multiply_half(y, upper);
        spread(reads_half_b, products_half);
        b0 = b1;
      }
      five(buf);
      multiply_half(y, upper);
    }
  }
  // An MFMA tile's lane holds m = lane % 16 and n = 4 (lane / 16) .. + 3.  Each
  // wave turns 64 rows at a time in LDS of its own, so that a lane then holds 8
  // neighbours of a row and rows are read and written in whole runs.  Quad q
  // (4 values) of row r lies at position q ^ (r & 15).  (The loop over the rows
  // must unroll: accumulators indexed at run time would live in scratch memory.)
  constexpr int kCols = BN / WN, kEights = kCols / 8, kQuads = kCols / 4;
  static_assert(kCols == 64 && kFm % 4 == 0 && kWaves * 64 * kCols * 4 <= (int)sizeof(lds), "epilogue buffers");
  floatx4* turn = reinterpret_cast<floatx4*>(&lds[0][0]) + wave * 64 * kQuads;
  __syncthreads();  // every wave has read its last tiles
#pragma unroll
  for (int i0 = 0; i0 < kFm; i0 += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kFn; ++j) {
        const int r = 16 * i + (lane & 15), q = 4 * j + (lane >> 4);
        turn[r * kQuads + (q ^ (r & 15))] = acc[i0 + i][j];
      }
    wave_fence();
    with_act<KIND>(g.act, [&](auto act) {
#pragma unroll 1
      for (int r = lane / kEights; r < 64; r += 64 / kEights) {
        const int c = lane % kEights;
        const floatx4 lo = turn[r * kQuads + ((2 * c) ^ (r & 15))], hi = turn[r * kQuads + ((2 * c + 1) ^ (r & 15))];
        const int64_t m = m0 + wm + 16 * i0 + r, n = n0 + wn + 8 * c;
        if (m < g.M && n < g.N) {
          if (g.splits > 1) {
            float* p = g.part + ((int64_t)blockIdx.y * g.M + m) * g.pn + n;
            *reinterpret_cast<floatx4*>(p) = lo;
            *reinterpret_cast<floatx4*>(p + 4) = hi;
          } else {
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            finish8<KIND, decltype(act)::value>(g, m, n, v);
          }
        }
      }
    });
    wave_fence();
  }
}

// The splits' partial sums and the epilogue: 64 outputs of 8 columns per block,
// each wave sums every fourth split (so that their loads are in flight
// together), wave 0 joins the four in order.  Bound by reading the partial sums
// (three of 384 x 7168: 8 us for 44 MB in and out, 5.4 TB/s from the caches).
template <int KIND>
__global__ __launch_bounds__(256) void k_linear_join(LinearGemm g) {
  __shared__ floatx4 red[3][2][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t eights = g.pn / 8, i = (int64_t)blockIdx.x * 64 + lane, step = g.M * g.pn;
  const bool in = i < g.M * eights;
  const int64_t m = i / eights, n = (i - m * eights) * 8;
  const float* p = g.part + m * g.pn + n;
  floatx4 lo = {}, hi = {};
  if (in) {
#pragma unroll 8
    for (int s = wave; s < g.splits; s += 4) {
      lo += *reinterpret_cast<const floatx4*>(p + s * step);
      hi += *reinterpret_cast<const floatx4*>(p + s * step + 4);
    }
  }
  if (wave) {
    red[wave - 1][0][lane] = lo;
    red[wave - 1][1][lane] = hi;
  }
  __syncthreads();
  if (wave || !in) return;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    lo += red[q][0][lane];
    hi += red[q][1][lane];
  }
  float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  with_act<KIND>(g.act, [&](auto act) { finish8<KIND, decltype(act)::value>(g, m, n, v); });
}

// ---------------------------------------------------------------- few rows

// The forward for up to 16 MT tokens, which is bound by reading the weight once:
// a block computes `cols` (4, 8 or 16) output columns for all tokens.  Its 16
// waves deal the contraction's 64-value pieces out in turn, read weight and
// inputs straight into fragments (32 bytes of a row per lane: a wave reads whole
// 128-byte lines of 16 rows; lanes past the last column or token repeat it), and
// their sums are joined through LDS in the waves' order.  One launch, no workspace.
// One token through 7168 x 384 takes 6.7 us, six of them latency (launch, two
// rounds of loads, the join): the weight's 5.5 MB alone are 1.1 us.
template <int MT>
__global__ __launch_bounds__(1024) void k_linear_few(LinearGemm g, int cols) {
  constexpr int kWaves = 16, kUnroll = MT == 1 ? 4 : MT == 2 ? 2 : 1;
  __shared__ float red[kWaves][MT][16 * 17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * cols;
  const int64_t n = min(n0 + min(j, cols - 1), g.N - 1);
  const uint16_t* pw = g.b + n * g.ldb + 16 * q;
  const uint16_t* px[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) px[i] = g.a + min((int64_t)(16 * i + j), g.M - 1) * g.lda + 16 * q;
  floatx4 acc[MT] = {};
  const int full = (int)(g.K / 64), pieces = (int)((g.K + 63) / 64);
  auto step = [&](int b, auto count) {
    constexpr int U = decltype(count)::value;
    u32x4 w[U][2], x[U][MT][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = (int64_t)(b + u * kWaves) * 64 + 8 * h;
        w[u][h] = *reinterpret_cast<const u32x4*>(pw + k);
#pragma unroll
        for (int i = 0; i < MT; ++i) x[u][i][h] = *reinterpret_cast<const u32x4*>(px[i] + k);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = mfma_bf16(w[u][h], x[u][i][h], acc[i]);
  };
  int b = wave;
  for (; b + (kUnroll - 1) * kWaves < full; b += kUnroll * kWaves) step(b, std::integral_constant<int, kUnroll>());
  for (; b < full; b += kWaves) step(b, std::integral_constant<int, 1>());
  if (b == full && full < pieces) {  // the last piece is short: values past K are zeros
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = (int64_t)full * 64 + 8 * h;
      const bool in = k + 16 * q < g.K;
      const u32x4 w = in ? *reinterpret_cast<const u32x4*>(pw + k) : u32x4{};
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = mfma_bf16(w, in ? *reinterpret_cast<const u32x4*>(px[i] + k) : u32x4{}, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][i][(4 * q + r) * 17 + j] = acc[i][r];
  __syncthreads();
  const int c = threadIdx.x & 15, m = threadIdx.x >> 4;
  if (m >= g.M || m >= 16 * MT || c >= cols || n0 + c >= g.N) return;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) v += red[k][m >> 4][c * 17 + (m & 15)];
  with_act<kLinFwd>(g.act, [&](auto act) { finish1<kLinFwd, decltype(act)::value>(g, m, n0 + c, v); });
}

// ---------------------------------------------------------------- dz and its column sums

// dz = grad_output * act'(preact) as bf16 planes that sum to it: p0 + p1 + p2 (24
// bits: dz itself, for |dz| above 2^-100) for d_weight, p0 + rest (2^-16 of dz: far
// below the rounding of the bf16 result) for grad_input, whose rounding to bf16
// would else not be its only one.
//
// The parts of a nonzero dz all have its sign and none is 0, so that they
// times an infinity give what dz times it is: with parts of both signs, or
// zeros, its product would be NaN.  So p0 and p1 are cut off, not rounded, and go
// a step towards 0 where they would leave nothing; the next part is then that step.
struct DzArgs {
  const void* dy;
  int dy_f32;
  const uint16_t* z;
  int act;
  int64_t T, N, pitch;  // planes are [T][pitch], zeros from N on
  uint16_t* plane;      // p0
  int64_t plane_size;   // elements from one plane to the next
  int planes;           // p0 alone (1), or with p1 and p2 (kMaxPlanes)
  int rest;             // which plane is p0's rest (0: none)
  float* part;          // [row blocks][N] column sums
};

__device__ __forceinline__ float dz_of(int act, float dy, float z) {
  if (act == KT_ACT_NONE) return dy;
  if (act == KT_ACT_RELU) return z > 0.f ? dy : z != z ? z : 0.f;
  return dy * act_slope(act, z);
}

// v's leading 8 bits, less a step where that is all of v.  (Selects, not branches: values of all kinds share a wave.)
__device__ __forceinline__ uint32_t cut_part(float v) {
  const uint32_t b = __float_as_uint(v), h = b >> 16, mag = b & 0x7fffffffu;
  const uint32_t step = (b & 0xffffu) == 0 && mag - 1 < 0x7f7fffffu;  // nonzero, finite
  return mag > 0x7f800000u ? h | 0x40u : h - step;                   // (a NaN stays one)
}

// What v's part h leaves; an infinity or a NaN stays whole.
__device__ __forceinline__ float left_by(float v, uint32_t h) {
  return (h & 0x7f80u) == 0x7f80u ? v : v - __uint_as_float(h << 16);
}

// p0, p1, p2 and the rest of p0 rounded to bf16.  p2 holds all that is left, so
// its cut loses nothing; a NaN's later parts may be anything beside p0.
__device__ __forceinline__ void split_planes(float v, uint16_t (&p)[kMaxPlanes + 1]) {
  const uint32_t h0 = cut_part(v);
  const float r0 = left_by(v, h0);
  const uint32_t h1 = cut_part(r0);
  p[0] = (uint16_t)h0;
  p[1] = (uint16_t)h1;
  p[2] = (uint16_t)(__float_as_uint(left_by(r0, h1)) >> 16);
  const uint32_t r = __float_as_uint(r0);
  p[3] = (uint16_t)((r + 0x7fffu + (r >> 16 & 1u)) >> 16);
}

constexpr int kDzRows = 32, kDzCols = 256;

// kDzCols columns x kDzRows rows per block, 8 columns a thread.  WIDE: N is a
// multiple of 8, so that a thread's values are 16-byte pieces.  Bound by memory:
// 8192 x 2048 with an activation and four planes moves 201 MB in 50 us (4.0 TB/s).
template <bool WIDE>
__global__ __launch_bounds__(256) void k_linear_dz(DzArgs a) {
  __shared__ float red[8][kDzCols + 4];
  const int c = (threadIdx.x & 31) * 8, q = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * kDzCols + c;
  float sum[8] = {};
  if (n < a.pitch) {
#pragma unroll
    for (int r = 0; r < kDzRows / 8; ++r) {
      const int64_t t = (int64_t)blockIdx.y * kDzRows + r * 8 + q;
      if (t >= a.T) break;
      const int64_t i = t * a.N + n;
      float v[8], z[8];
      if (WIDE) {
        if (a.dy_f32) {
          const floatx4* p = reinterpret_cast<const floatx4*>(static_cast<const float*>(a.dy) + i);
          const floatx4 lo = p[0], hi = p[1];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = k < 4 ? lo[k & 3] : hi[k & 3];
        } else {
          const u32x4 p = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.dy) + i);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = bf16_to_float((uint16_t)(p[k >> 1] >> (16 * (k & 1))));
        }
        if (a.act != KT_ACT_NONE) {
          const u32x4 p = *reinterpret_cast<const u32x4*>(a.z + i);
#pragma unroll
          for (int k = 0; k < 8; ++k) z[k] = bf16_to_float((uint16_t)(p[k >> 1] >> (16 * (k & 1))));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool in = n + k < a.N;
          v[k] = !in        ? 0.f
                 : a.dy_f32 ? static_cast<const float*>(a.dy)[i + k]
                            : bf16_to_float(static_cast<const uint16_t*>(a.dy)[i + k]);
          if (a.act != KT_ACT_NONE) z[k] = in ? bf16_to_float(a.z[i + k]) : 0.f;
        }
      }
      if (a.act != KT_ACT_NONE) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = dz_of(a.act, v[k], z[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += v[k];
      if (a.plane) {
        uint16_t p[8][kMaxPlanes + 1];
        const bool whole = a.planes == 1 && !a.rest;  // bf16 holds every v: p0 is v
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (whole)
            p[k][0] = float_to_bf16(v[k]);
          else
            split_planes(v[k], p[k]);
        }
        auto put = [&](int w, int to) {
          *reinterpret_cast<u32x4*>(a.plane + to * a.plane_size + t * a.pitch + n) =
              u32x4{pack2(p[0][w], p[1][w]), pack2(p[2][w], p[3][w]), pack2(p[4][w], p[5][w]), pack2(p[6][w], p[7][w])};
        };
        put(0, 0);
        if (a.planes > 1) {
          put(1, 1);
          put(2, 2);
        }
        if (a.rest) put(3, a.rest);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) red[q][c + k] = sum[k];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * kDzCols + threadIdx.x;
  if (col < a.N) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][threadIdx.x];
    a.part[(int64_t)blockIdx.y * a.N + col] = s;
  }
}

// Column sums of the row blocks' parts: 64 columns x 16 runs of parts per block.
__global__ __launch_bounds__(1024) void k_linear_db(const float* __restrict__ part, int64_t nb, int64_t N,
                                                    float* __restrict__ db, int accumulate, float scale) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 64 + c;
  float s = 0.f;
  if (n < N) {
#pragma unroll 4
    for (int64_t b = q; b < nb; b += 16) s += part[b * N + n];
  }
  red[q][c] = s;
  __syncthreads();
  if (q || n >= N) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += red[k][c];
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

// How a product runs.
//   few      forward of few tokens: k_linear_few.  7168 x 384: 6.7 us for one token, 11.2 for 16, where tiles
//            with their splits and joining launch take 11.1 us for 32 and no less for fewer; 2048 x 7168:
//            10.1 us for 16 tokens against 15; 512 x 384: 4.4 us for 64 against 8.3.  It reads the inputs once
//            per block, so it loses where tokens and K are large (7168 x 384, 64 tokens: 30 against 11.7 us).
//   big      256 x 256 tiles, where they fill three quarters of the chip (two rows of fragments then serve
//            twice the MFMAs).  Forward of 8192 x 7168 x 2048: 1.27 against 1.14 PFLOP/s with 128 x 128
//            tiles, d_weight 1.21 against 1.02 (three planes: 1.26 against 1.14), grad_input of 16384 x 2048
//            from a contraction of 7168 1.25 against 1.04; of 8192 x 7168 from 2048 the same, and within 5% at
//            contractions of 384 (forward 83 against 87 us, grad_input 68 against 67, 133 against 135).  With
//            fewer: 4096 x 2048 x 2048 (128 of them) 56 us against 38.
//   splits   of the contraction, where 128 x 128 tiles alone leave units without the two blocks they can
//            hold: as many as give 512 blocks (d_weight of 4096 x 7168 x 384 with three planes: 114 us with
//            1, 89 with 2, 77 with 3 and 89 with 4), each with at least four steps, or eight above 64 rows,
//            where the partial sums cost more (2048 x 2048, 512 tokens: 21 us with 4 splits of 8 steps, 25 with
//            8 of 4; 7168 x 384, 32 tokens: 11 us with 28 splits of 4 steps, 13 with 14 of 8).
constexpr int kBlocksWanted = 512, kMaxSplits = 64;

struct LinearShape {
  int few;   // 16-row tiles of k_linear_few (0: not used)
  bool big;
  int64_t tiles;
  int splits;
};

// planes: of A
static LinearShape linear_shape(LinearKind kind, int64_t M, int64_t N, int64_t K, int planes) {
  LinearShape s{};
  s.splits = 1;
  if (kind == kLinFwd && (M <= 16 || (M <= 64 && M * K <= 65536))) {
    s.few = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    return s;
  }
  const int step = linear_step(kind == kLinDw ? planes : 1);
  const int64_t steps = (K + step - 1) / step * (kind == kLinDx ? planes : 1);
  const int64_t big = (M + 255) / 256 * ((N + 255) / 256);
  s.big = big >= 192;
  s.tiles = s.big ? big : (M + 127) / 128 * ((N + 127) / 128);
  int64_t splits = s.big || s.tiles == 0 ? 1 : kBlocksWanted / s.tiles;
  const int64_t least = M <= 64 ? 4 : 8;
  if (splits > steps / least) splits = steps / least;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits > 1) s.splits = (int)splits;
  return s;
}

static int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

static size_t part_bytes(const LinearShape& s, int64_t M, int64_t N) {
  return s.splits > 1 ? round256(4 * (size_t)s.splits * (size_t)M * (size_t)round_up(N, 8)) : 0;
}

// The most that part_bytes is for 1 .. T rows: fewer rows may take more splits.
// Between multiples of 128 rows, and above and below 64, the splits stay.
static size_t most_part_bytes(LinearKind kind, int64_t T, int64_t N, int64_t K, int planes) {
  auto bytes = [&](int64_t M) { return part_bytes(linear_shape(kind, M, N, K, planes), M, N); };
  size_t most = bytes(T);
  if (T > 64) most = std::max(most, bytes(64));
  // over kBlocksWanted / 2 tiles nothing is split
  for (int64_t M = 128; M < T && M / 128 * ((N + 127) / 128) <= kBlocksWanted / 2; M += 128) most = std::max(most, bytes(M));
  return most;
}

// The workspace of a backward.  Every part has room of its own except the
// splits' partial sums, which the two products use one after the other.
struct LinearBwdPlan {
  LinearShape dx, dw;
  size_t planes, part, db, x, total;
  int64_t pitch, nb;
};

// most: at its largest for 1 .. T tokens
static LinearBwdPlan plan_linear_bwd(const kt_linear* L, int64_t T, bool ckpt, bool most = false) {
  LinearBwdPlan p{};
  const int64_t N = L->out_features, K = L->in_features;
  p.pitch = round_up(N, 8);
  p.nb = (T + kDzRows - 1) / kDzRows;
  // (with one plane no more splits)
  p.dx = linear_shape(kLinDx, T, K, N, kDxPlanes);
  p.dw = linear_shape(kLinDw, N, K, T, kMaxPlanes);
  p.planes = 0;
  p.db = p.planes + round256(2 * (kMaxPlanes + 1) * (size_t)T * (size_t)p.pitch);
  p.part = p.db + round256(4 * (size_t)p.nb * (size_t)N);
  const size_t a = most ? most_part_bytes(kLinDx, T, K, N, kDxPlanes) : part_bytes(p.dx, T, K);
  p.x = p.part + std::max(a, part_bytes(p.dw, N, K));  // (d_weight's splits grow with T)
  p.total = p.x + (ckpt ? round256(2 * (size_t)T * (size_t)K) : 0);
  return p;
}

template <int KIND, int PLANES = 1>
static void launch_linear(LinearGemm g, const LinearShape& s, float* part, hipStream_t st) {
  g.splits = s.splits;
  g.part = part;
  g.pn = round_up(g.N, 8);
  if constexpr (KIND == kLinFwd) {
    if (s.few) {
      // narrower blocks fill more of the chip, wider ones read the inputs less often (7168 x 384: 6.7, 7.6
      // and 9.9 us with 4, 8 and 16; 7168 x 2048: 13.7, 9.4, 11.6; 2048 x 7168: 14.5, 10.5, 8.2)
      const int cols = g.N >= 4096 ? 16 : g.N >= 1024 ? 8 : 4;
      const unsigned blocks = (unsigned)((g.N + cols - 1) / cols);
      if (s.few == 1)
        k_linear_few<1><<<blocks, 1024, 0, st>>>(g, cols);
      else if (s.few == 2)
        k_linear_few<2><<<blocks, 1024, 0, st>>>(g, cols);
      else
        k_linear_few<4><<<blocks, 1024, 0, st>>>(g, cols);
      note_launch();
      return;
    }
  }
  const dim3 grid((unsigned)s.tiles, (unsigned)s.splits);
  if (s.big)
    k_linear<KIND, 256, 256, 2, 4, PLANES><<<grid, 512, 0, st>>>(g);
  else
    k_linear<KIND, 128, 128, 2, 2, PLANES><<<grid, 256, 0, st>>>(g);
  note_launch();
  if (s.splits > 1) {
    k_linear_join<KIND><<<(unsigned)((g.M * (g.pn / 8) + 63) / 64), 256, 0, st>>>(g);
    note_launch();
  }
}

}  // namespace kt

using namespace kt;

extern "C" {

size_t kt_linear_workspace_bytes(const kt_linear* linear, int32_t tokens) {
  if (check_linear(linear, tokens)) return 0;
  (void)set_error(KT_RAWINT4_OK, "");  // 0 is a valid size: no message stays
  return most_part_bytes(kLinFwd, tokens, linear->out_features, linear->in_features, 1);
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
  const LinearShape s = linear_shape(kLinFwd, tokens, N, K, 1);
  const size_t need = part_bytes(s, tokens, N);
  if (need) {
    rc = check_caller_workspace(workspace, workspace_bytes, need);
    if (rc) return rc;
  }
  if (tokens == 0) return set_error(KT_RAWINT4_OK, "");
  begin_launches();
  LinearGemm g{};
  g.a = inputs;
  g.lda = K;
  g.b = linear->weight;
  g.ldb = K;
  g.M = tokens;
  g.N = N;
  g.K = K;
  g.bias = linear->bias;
  g.residual = residual;
  g.out = output;
  g.out_f32 = output_type == KT_TYPE_F32;
  g.preact = preact;
  g.act = linear->activation;
  launch_linear<kLinFwd>(g, s, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
  return finish_launches();
}

size_t kt_linear_bwd_workspace_bytes(const kt_linear* linear, int32_t tokens, int32_t from_checkpoint) {
  if (check_linear(linear, tokens)) return 0;
  (void)set_error(KT_RAWINT4_OK, "");
  return plan_linear_bwd(linear, tokens, from_checkpoint != 0, true).total;
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
    if (!accumulate && d_weight) {
      const int64_t most = (int64_t)1 << 31;  // N K may be 2^32, more threads than a launch takes
      for (int64_t i = 0; i < N * K; i += most)
        launch_fill_zero_f32(d_weight + i, N * K - i < most ? N * K - i : most, st);
    }
    if (!accumulate && d_bias) launch_fill_zero_f32(d_bias, N, st);
    return finish_launches();
  }
  const LinearBwdPlan p = plan_linear_bwd(linear, T, checkpoint != nullptr);
  rc = check_caller_workspace(workspace, workspace_bytes, p.total);
  if (rc) return rc;
  begin_launches();
  // a bf16 grad_output without activation is dz itself (its rows must start at 16 bytes)
  const bool exact = !act && grad_output_type == KT_TYPE_BF16, products = grad_input || d_weight;
  const bool direct = (exact && N % 8 == 0) || !products;
  const uint16_t* dz = static_cast<const uint16_t*>(grad_output);
  const int64_t pitch = direct ? N : p.pitch;
  const int planes = exact || !d_weight ? 1 : kMaxPlanes, rest = exact || !grad_input ? 0 : planes;
  if (!direct || d_bias) {
    DzArgs a{};
    a.dy = grad_output;
    a.dy_f32 = grad_output_type == KT_TYPE_F32;
    a.z = preact;
    a.act = linear->activation;
    a.T = T;
    a.N = N;
    a.pitch = p.pitch;
    a.plane = direct ? nullptr : ws_ptr<uint16_t>(workspace, p.planes);
    a.plane_size = T * p.pitch;
    a.planes = planes;
    a.rest = rest;
    a.part = d_bias ? ws_ptr<float>(workspace, p.db) : nullptr;
    const dim3 grid((unsigned)((p.pitch + kDzCols - 1) / kDzCols), (unsigned)p.nb);
    if (N % 8 == 0)
      k_linear_dz<true><<<grid, 256, 0, st>>>(a);
    else
      k_linear_dz<false><<<grid, 256, 0, st>>>(a);
    note_launch();
    if (!direct) dz = a.plane;
    if (d_bias) {
      k_linear_db<<<(unsigned)((N + 63) / 64), 1024, 0, st>>>(a.part, p.nb, N, d_bias, accumulate, grad_scale);
      note_launch();
    }
  }
  LinearGemm g{};
  if (grad_input) {
    g.a = dz;
    g.lda = pitch;
    g.b = linear->weight;
    g.ldb = K;
    g.M = T;
    g.N = K;
    g.K = N;
    g.a_plane = rest * T * p.pitch;
    g.planes = rest ? kDxPlanes : 1;
    g.residual = grad_residual;
    g.out = grad_input;
    launch_linear<kLinDx>(g, linear_shape(kLinDx, T, K, N, g.planes), ws_ptr<float>(workspace, p.part), st);
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
    g.lda = pitch;
    g.a_width = pitch;
    g.b = x;
    g.ldb = K;
    g.M = N;
    g.N = K;
    g.K = T;
    g.a_plane = T * p.pitch;
    g.out = d_weight;
    g.accumulate = accumulate;
    g.scale = grad_scale;
    const LinearShape s = linear_shape(kLinDw, N, K, T, planes);
    if (planes == 1)
      launch_linear<kLinDw>(g, s, ws_ptr<float>(workspace, p.part), st);
    else
      launch_linear<kLinDw, kMaxPlanes>(g, s, ws_ptr<float>(workspace, p.part), st);
  }
  return finish_launches();
}

}  // extern "C"
