// The routed experts for a few tokens (decoding): gate and up in one kernel,
// down with the weighted sum over the slots in another, two small ones more with LoRA.
//
// With few tokens an expert has one or two of them, and the time is that of
// reading its packed rows once.  Weights go into the MFMAs as bf16, one MFMA
// (32 contraction values) per 16 weight rows and scale group, so that the
// scale multiplies the group's sum in fp32.
//   RAWINT4: a code c becomes 1 + c / 16, by a shift and an and-or for two of
//   them, exact in bf16, and
//     sum (c - 8) x = 16 (sum (1 + c / 16) x - 3/2 sum x),
//   where -3/2 sum x of the group is the MFMA's initial sum (an MFMA of x with
//   -3/2).  Products are exact, whatever the inputs' and scales' size.
//   MXFP4: a code is converted to bf16 as it is, the initial sum is 0.
// Inputs are bf16 as given; h, fp32, enters as two bf16 (hi and lo), 2^-16 of
// it left out.
//
// The other operand's 16 rows are four vectors (tokens, or hi and lo of two)
// by four scale groups: 16 bytes a lane bring 128 contraction values of all
// four, and of the MFMA with group j's weights the rows of group j are
// taken, register j of every lane.  So x and h need no staging: they come from
// the caches in the same stream of loads as the codes, and no workgroup
// waits for another's.  A lane loads 16 bytes of a weight row, a whole scale
// group; an exchange of 4 x 4 dwords between the wave's four rows of 16 lanes
// gives each MFMA one group.
#include "kt_step_common.hpp"

#include <math.h>

namespace kt {

struct DecodeArgs {
  int S, k, T;  // slots, slots a token, tokens
  int E, H, I, R;
  float sc, limit;
  const uint16_t* x;
  const int64_t* ids;
  const float* rw;
  uint16_t* out;
  const uint8_t *wg, *wu, *wd;
  const uint16_t *sg, *su, *sd;
  const float *ag, *bg, *au, *bu, *ad, *bd;
  float* h;       // [S][I], with LoRA
  uint16_t* hs;   // [S][2][I]: h as bf16 hi and lo, in the codes' order
  int32_t* next;  // [S]: the next slot of the same expert, -1 for none
  int32_t* lead;  // [S]: whether the slot is its expert's first
  float* ua;      // [S][2 R]: x A_g^T | x A_u^T
  float* ud;      // [S][R]: h A_d^T
};

typedef u32x4 u32x4_u2 __attribute__((aligned(2)));

// The slots of slot `s`'s expert e from s on, in order, to list[] (wave 0
// writes; every wave finds the same number); 0 if another slot comes before.
// `next`: the slot after s, or -1.
__device__ __forceinline__ int slots_of(const DecodeArgs& a, int s, int64_t e, uint16_t* list, int& next) {
  const int lane = threadIdx.x & 63;
  next = -1;
  int n = 0;
  bool led = false;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const bool hit = s0 + lane < a.S && a.ids[s0 + lane] == e;
    const uint64_t mask = __ballot(hit);
    const uint64_t upto = s - s0 >= 63 ? ~0ull : s < s0 ? 0ull : (2ull << (s - s0)) - 1;  // slots <= s of these 64
    const uint64_t own = s >= s0 && s - s0 < 64 ? 1ull << (s - s0) : 0ull;
    led |= (mask & upto & ~own) != 0;
    const uint64_t rest = mask & ~(upto & ~own);
    if (hit && (rest >> lane & 1) && threadIdx.x < 64) list[n + __popcll(rest & ((1ull << lane) - 1))] = (uint16_t)(s0 + lane);
    n += __popcll(rest);
    if (next < 0 && (rest & ~own)) next = s0 + __ffsll((unsigned long long)(rest & ~own)) - 1;
  }
  return led ? 0 : n;
}

// Registers r[0..3] of a lane in row q hold the 16 bytes (dwords 0..3) of group q; afterwards r[i] is dword q of group i.
__device__ __forceinline__ void transpose4(uint32_t* r) {
  swap32(r[0], r[2]);
  swap32(r[1], r[3]);
  swap16(r[0], r[1]);
  swap16(r[2], r[3]);
}

// 8 codes of a dword as bf16: RAWINT4 1 + c / 16 in the order k0 k4 k1 k5 k2 k6 k3 k7, MXFP4 their values in order.
template <bool MX>
__device__ __forceinline__ u32x4 codes_bf16(uint32_t w) {
  if (MX) {
    auto two = [&](auto sel) {
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, decltype(sel)::value));
    };
    return u32x4{two(std::integral_constant<int, 0>()), two(std::integral_constant<int, 1>()),
                 two(std::integral_constant<int, 2>()), two(std::integral_constant<int, 3>())};
  }
  const uint32_t m = 0x00780078u, o = 0x3f803f80u;
  return u32x4{((w << 3) & m) | o, ((w >> 1) & m) | o, ((w >> 5) & m) | o, ((w >> 9) & m) | o};
}

// 8 bf16 in order -> the order of codes_bf16<false>
__device__ __forceinline__ u32x4 order8(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
               __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Loads through a buffer descriptor: a base and an offset that are the same in
// all lanes, and the lane's 32-bit offset.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 buffer16(Buffer b, uint32_t lane, uint32_t base) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane, (int)base, 0));
}

// A contraction goes in units of 256 values (8 scale groups).  Every load is
// issued, whatever the unit, so that how many are in flight behind a value is
// known where it is waited for; those of a unit that reaches past the
// contraction (of G groups) are moved to where they stay inside their matrix,
// and what they bring is not used (`trim`).
//
// A unit of 16 weight rows, this lane's share: codes of groups q and 4 + q of row n, and the row's 8 scales.
struct Codes {
  u32x4 c[2], s;
};
// Where a lane's share lies in an expert's matrix: codes from unit 0 on, those of a unit past the end, the
// scales, and the last 16 bytes of scales.
struct Place {
  uint32_t w, end[2], s, last;
};
__device__ __forceinline__ Place place_of(int rows, int row, int G, int q) {
  const uint32_t pitch = (uint32_t)G * 16, first = (uint32_t)row * pitch + q * 16, most = (uint32_t)rows * pitch - 16;
  const uint32_t tail = first + (uint32_t)(G / 8) * 128;
  return {first, {min(tail, most), min(tail + 64, most)}, (uint32_t)row * (uint32_t)G * 2, (uint32_t)rows * (uint32_t)G * 2 - 16};
}
struct Matrix {  // of one expert
  Buffer w;
  const uint8_t* s;
};
__device__ __forceinline__ Matrix matrix_of(const uint8_t* w, const uint16_t* s, size_t e, int rows, int G) {
  const size_t n = (size_t)rows * G;
  return {buffer_of(w + e * n * 16, n * 16), reinterpret_cast<const uint8_t*>(s + e * n)};
}
__device__ __forceinline__ void load_codes(const Matrix& m, const Place& p, int u, bool past, Codes& c) {
  c.c[0] = buffer16(m.w, past ? p.end[0] : p.w, past ? 0 : (uint32_t)u * 128);
  c.c[1] = buffer16(m.w, past ? p.end[1] : p.w + 64, past ? 0 : (uint32_t)u * 128);
  c.s = *reinterpret_cast<const u32x4_u2*>(m.s + min(p.s + (uint32_t)u * 16, p.last));
}
// scales of groups behind G are 0
__device__ __forceinline__ void trim(const Place& p, int u, int G, Codes& c) {
  const uint32_t at = p.s + (uint32_t)u * 16, d = at > p.last ? (at - p.last) / 2 : 0;  // scales that came before the unit's
  uint32_t w[4] = {c.s.x, c.s.y, c.s.z, c.s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = d & 1 ? (w[i] >> 16 | (i < 3 ? w[i + 1] << 16 : 0)) : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = d & 2 ? (i < 3 ? w[i + 1] : 0) : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = d & 4 ? (i < 2 ? w[i + 2] : 0) : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = 8 * u + 2 * i;
    c.s[i] = g + 1 < G ? w[i] : g < G ? w[i] & 0xffffu : 0u;
  }
}

// The vectors' share of a unit: of the lane's vector (n / 4) and group n % 4 the 8 values from 8 q on.
struct Vecs {
  u32x4 v[2];
};
struct VecPlace {
  uint32_t v, end[2];
};
__device__ __forceinline__ VecPlace vec_place(uint32_t vec, uint32_t vecs, int G, int n, int q) {
  const uint32_t first = (vec * (uint32_t)G * 32 + (n & 3) * 32 + q * 8) * 2, most = vecs * (uint32_t)G * 64 - 16;
  const uint32_t tail = first + (uint32_t)(G / 8) * 512;
  return {first, {min(tail, most), min(tail + 256, most)}};
}
__device__ __forceinline__ void load_vecs(Buffer b, const VecPlace& p, int u, bool past, Vecs& x) {
  x.v[0] = buffer16(b, past ? p.end[0] : p.v, past ? 0 : (uint32_t)u * 512);
  x.v[1] = buffer16(b, past ? p.end[1] : p.v + 256, past ? 0 : (uint32_t)u * 512);
}
__device__ __forceinline__ void trim(int u, int G, int n, Vecs& x) {
  const u32x4 zero = {0, 0, 0, 0};
  if (8 * u + (n & 3) >= G) x.v[0] = zero;
  if (8 * u + 4 + (n & 3) >= G) x.v[1] = zero;
}

// The MFMAs' initial sums for four groups of the vectors.
template <bool MX>
__device__ __forceinline__ floatx4 initial(const u32x4& x) {
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  return MX ? zero : mfma_bf16(x, u32x4{0xbfc0bfc0u, 0xbfc0bfc0u, 0xbfc0bfc0u, 0xbfc0bfc0u}, zero);
}

// Adds half i of the codes' values times the vectors to this lane's sum (weight row n, vector q).
template <bool MX>
__device__ __forceinline__ void multiply(const Codes& c, int i, const u32x4& x, const floatx4& init, float& acc) {
  uint32_t r[4] = {c.c[i].x, c.c[i].y, c.c[i].z, c.c[i].w};
  transpose4(r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t s = c.s[2 * i + j / 2];
    acc = fmaf(j & 1 ? bf_hi(s) : bf_lo(s), mfma_bf16(x, codes_bf16<MX>(r[j]), init)[j], acc);
  }
  __builtin_amdgcn_sched_barrier(0);  // (more MFMAs side by side take registers from the loads ahead)
}

constexpr int kVecs = 4;      // tokens that gate and up take at a time
constexpr int kLoraParts = 8;  // runs of the ranks

// Gate and up.  A workgroup has 16 columns of I of one expert (its first
// slot's block; the others leave at once) for all of its tokens, four at a time.
// Its four waves split the contraction.
template <bool MX, bool LORA>
__global__ __launch_bounds__(256, 3) void k_decode_gate_up(DecodeArgs a) {
  __shared__ uint16_t list[KT_MOE_DECODE_MAX_SLOTS];
  __shared__ float red[2][4][kVecs][16];
  __shared__ float lora[LORA ? kLoraParts : 1][2][kVecs][16];
  const int slot = blockIdx.y, i0 = blockIdx.x * 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t e = a.ids[slot];
  int next = -1, M = 0;
  if (e >= 0 && e < a.E) M = slots_of(a, slot, e, list, next);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.next[slot] = next;
    a.lead[slot] = M > 0;
  }
  if (!M) return;
  const int G = a.H / 32, units = (G + 7) / 8, per = (units + 3) / 4, kw = __builtin_amdgcn_readfirstlane(wave);
  const int u0 = kw * per;
  const Matrix mg = matrix_of(a.wg, a.sg, e, a.I, G), mu = matrix_of(a.wu, a.su, e, a.I, G);
  const Place at = place_of(a.I, i0 + n, G, q);
  const Buffer xb = buffer_of(a.x, (size_t)a.T * a.H * 2);
  __syncthreads();
  for (int m0 = 0; m0 < M; m0 += kVecs) {
    const int nt = min(kVecs, M - m0);
    const VecPlace xat = vec_place(list[m0 + min(n >> 2, nt - 1)] / a.k, a.T, G, n, q);
    float g = 0.f, u = 0.f;
    Codes cg[2], cu[2];
    Vecs xv[2];
    auto load = [&](int v, int b) {
      const bool past = 8 * v + 8 > G;
      load_codes(mg, at, v, past, cg[b]);
      load_codes(mu, at, v, past, cu[b]);
      load_vecs(xb, xat, v, past, xv[b]);
      asm volatile("" ::: "memory");  // (loads stay here, in this order)
    };
    load(u0, 0);
    load(u0 + 1, 1);
    if (LORA) {
      // columns by gate and up by runs of the ranks
      const int c = threadIdx.x & 15, up = threadIdx.x >> 4 & 1, part = threadIdx.x >> 5;
      const int len = (a.R + kLoraParts - 1) / kLoraParts, r0 = part * len, r1 = min(a.R, r0 + len);
      const float* b = (up ? a.bu : a.bg) + ((size_t)e * a.I + i0 + c) * a.R;
      float t[kVecs] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int r = r0; r < r1; ++r) {
        const float w = b[r];
#pragma unroll
        for (int p = 0; p < kVecs; ++p)
          if (p < nt) t[p] = fmaf(w, a.ua[(size_t)list[m0 + p] * 2 * a.R + up * a.R + r], t[p]);
      }
#pragma unroll
      for (int p = 0; p < kVecs; ++p) lora[part][up][p][c] = t[p];
    }
    for (int v = u0; v < u0 + per; v += 2) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (8 * (v + b) + 8 > G) {
          trim(at, v + b, G, cg[b]);
          trim(at, v + b, G, cu[b]);
          trim(v + b, G, n, xv[b]);
        }
        if (v + b < u0 + per) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const u32x4 x = MX ? xv[b].v[i] : order8(xv[b].v[i]);
            const floatx4 init = initial<MX>(x);
            multiply<MX>(cg[b], i, x, init, g);
            multiply<MX>(cu[b], i, x, init, u);
          }
        }
        load(v + b + 2, b);
      }
    }
    red[0][kw][q][n] = g;
    red[1][kw][q][n] = u;
    __syncthreads();
    if (threadIdx.x < 16 * nt) {
      const int p = threadIdx.x >> 4, c = threadIdx.x & 15;
      const float by = MX ? 1.f : 16.f;
      float gv = by * (red[0][0][p][c] + red[0][1][p][c] + red[0][2][p][c] + red[0][3][p][c]);
      float uv = by * (red[1][0][p][c] + red[1][1][p][c] + red[1][2][p][c] + red[1][3][p][c]);
      const int s = list[m0 + p];
      if (LORA) {
        float lg = 0.f, lu = 0.f;
#pragma unroll
        for (int r = 0; r < kLoraParts; ++r) lg += lora[r][0][p][c], lu += lora[r][1][p][c];
        gv = fmaf(a.sc, lg, gv), uv = fmaf(a.sc, lu, uv);
      }
      if (a.limit > 0.f) {
        // (comparisons that keep a NaN)
        gv = gv > a.limit ? a.limit : gv;
        uv = uv > a.limit ? a.limit : uv < -a.limit ? -a.limit : uv;
      }
      const float h = gv * sigmoid_f(gv) * uv;
      uint16_t hi, lo;
      split_bf16(h, hi, lo);
      uint16_t* o = a.hs + (size_t)s * 2 * a.I + i0 + (MX ? c : perm_pos(c));
      o[0] = hi;
      o[a.I] = lo;
      if (LORA) a.h[(size_t)s * a.I + i0 + c] = h;
    }
    if (m0 + kVecs < M) __syncthreads();
  }
}

// x A_g^T | x A_u^T of every slot (DOWN: h A_d^T): a wave per row of A of an expert, for all of its tokens, four at a time.
template <bool DOWN>
__global__ __launch_bounds__(256) void k_decode_lora_a(DecodeArgs a) {
  __shared__ uint16_t list[KT_MOE_DECODE_MAX_SLOTS];
  const int64_t e = a.ids[blockIdx.y];
  if (e < 0 || e >= a.E) return;
  int next;
  const int M = slots_of(a, blockIdx.y, e, list, next);
  if (!M) return;
  __syncthreads();
  const int rows = DOWN ? a.R : 2 * a.R, r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (r >= rows) return;
  const int K = DOWN ? a.I : a.H;
  const float* w = (DOWN ? a.ad : r < a.R ? a.ag : a.au) + ((size_t)e * a.R + (r < a.R ? r : r - a.R)) * K;
  for (int m0 = 0; m0 < M; m0 += kVecs) {
    const int nt = min(kVecs, M - m0);
    float v[kVecs] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = lane * 4; c < K; c += 256) {
      const float4 b = *reinterpret_cast<const float4*>(w + c);
#pragma unroll
      for (int p = 0; p < kVecs; ++p) {
        if (p >= nt) break;
        float4 x;
        if (DOWN) {
          x = *reinterpret_cast<const float4*>(a.h + (size_t)list[m0 + p] * K + c);
        } else {
          const u32pair t = *reinterpret_cast<const u32pair*>(a.x + (size_t)(list[m0 + p] / a.k) * K + c);
          x = float4{bf_lo(t.x), bf_hi(t.x), bf_lo(t.y), bf_hi(t.y)};
        }
        v[p] = fmaf(b.x, x.x, v[p]);
        v[p] = fmaf(b.y, x.y, v[p]);
        v[p] = fmaf(b.z, x.z, v[p]);
        v[p] = fmaf(b.w, x.w, v[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < kVecs; ++p) {
      const float t = wave_sum(v[p]);
      if (p < nt && lane == 0) (DOWN ? a.ud : a.ua)[(size_t)list[m0 + p] * rows + r] = t;
    }
  }
}

constexpr int kDownWaves = 8;
constexpr int kDownDepth = 3;  // units of loads ahead

// Down and the sum over the slots.  A workgroup has 16 columns of H; its waves
// take the experts in turn (a wave per expert, the whole contraction), two tokens at a
// time, and add to sums of their own per token, which the end joins in the waves' order.
template <bool MX, bool LORA>
__global__ __launch_bounds__(512, 4) void k_decode_down(DecodeArgs a) {
  extern __shared__ __align__(16) float acc[];  // [waves][T][16]
  __shared__ uint16_t order[KT_MOE_DECODE_MAX_SLOTS];
  __shared__ int16_t next[KT_MOE_DECODE_MAX_SLOTS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int h0 = blockIdx.x * 16, G = a.I / 32, units = (G + 7) / 8;
  const Place at = place_of(a.H, h0 + n, G, q);
  const Buffer hb = buffer_of(a.hs, (size_t)a.S * a.I * 4);
  int U = 0;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const bool lead = s0 + lane < a.S && a.lead[s0 + lane];
    const uint64_t mask = __ballot(lead);
    if (wave == 0) {
      if (s0 + lane < a.S) next[s0 + lane] = (int16_t)a.next[s0 + lane];
      if (lead) order[U + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)(s0 + lane);
    }
    U += __popcll(mask);
  }
  for (int i = threadIdx.x; i < kDownWaves * a.T * 16; i += 512) acc[i] = 0.f;
  __syncthreads();
  for (int j = wave; j < U; j += kDownWaves) {
    const int first = __builtin_amdgcn_readfirstlane(order[j]);
    const size_t e = (size_t)a.ids[first];
    const Matrix md = matrix_of(a.wd, a.sd, e, a.H, G);
    for (int s = first; s >= 0;) {
      const int s1 = __builtin_amdgcn_readfirstlane(next[s]);
      // vectors: hi and lo of slot s, hi and lo of slot s1
      const VecPlace hat = vec_place(((n >> 3) && s1 >= 0 ? s1 : s) * 2 + (n >> 2 & 1), 2 * a.S, G, n, q);
      Codes cd[kDownDepth];
      Vecs hv[kDownDepth];
      float y = 0.f;
      auto load = [&](int u, int b) {
        const bool past = 8 * u + 8 > G;
        load_codes(md, at, u, past, cd[b]);
        load_vecs(hb, hat, u, past, hv[b]);
        asm volatile("" ::: "memory");
      };
#pragma unroll
      for (int b = 0; b < kDownDepth; ++b) load(b, b);
      for (int u = 0; u < units; u += kDownDepth) {
#pragma unroll
        for (int b = 0; b < kDownDepth; ++b) {
          if (8 * (u + b) + 8 > G) {
            trim(at, u + b, G, cd[b]);
            trim(u + b, G, n, hv[b]);
          }
          if (u + b < units) {
#pragma unroll
            for (int i = 0; i < 2; ++i) multiply<MX>(cd[b], i, hv[b].v[i], initial<MX>(hv[b].v[i]), y);
          }
          load(u + b + kDownDepth, b);
        }
      }
      // hi + lo: rows of lanes 0 and 1 have slot s, 2 and 3 slot s1
      uint32_t y0 = __float_as_uint(y), y1 = y0;
      swap16(y0, y1);
      y = __uint_as_float(y0) + __uint_as_float(y1);
      if (!MX) y *= 16.f;
      const int mine = q < 2 ? s : s1;
      if (LORA) {
        // a quarter of the ranks a row of lanes
        const float* b = a.bd + (e * a.H + h0 + n) * a.R;
        float t0 = 0.f, t1 = 0.f;
#pragma unroll 1
        for (int r = q; r < a.R; r += 4) {
          t0 = fmaf(b[r], a.ud[(size_t)s * a.R + r], t0);
          if (s1 >= 0) t1 = fmaf(b[r], a.ud[(size_t)s1 * a.R + r], t1);
        }
        t0 = rows_sum(t0), t1 = rows_sum(t1);
        y = fmaf(a.sc, q < 2 ? t0 : t1, y);
      }
      // (both slots may be of one token)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (q == 2 * t && mine >= 0) {
          float* o = acc + (wave * a.T + mine / a.k) * 16 + n;
          *o = fmaf(a.rw[mine], y, *o);
        }
        wave_fence();
      }
      s = s1 >= 0 ? __builtin_amdgcn_readfirstlane(next[s1]) : -1;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += 512) {
    float v = 0.f;
    for (int w = 0; w < kDownWaves; ++w) v += acc[w * a.T * 16 + i];
    a.out[(size_t)(i >> 4) * a.H + h0 + (i & 15)] = float_to_bf16(v);
  }
}

// ---------------------------------------------------------------- host

struct DecodePlan {
  size_t hs, h, next, lead, ua, ud, total;
};
static DecodePlan plan_decode(const Dims& d) {
  DecodePlan p;
  const size_t S = (size_t)d.Ms;
  p.next = 0;
  p.lead = round256(4 * S);
  p.hs = p.lead + round256(4 * S);
  p.h = p.hs + round256(4 * S * d.I);
  p.ua = p.h + (d.R ? round256(4 * S * d.I) : 0);
  p.ud = p.ua + round256(4 * S * 2 * d.R);
  p.total = p.ud + round256(4 * S * d.R);
  return p;
}

static int check_decode(const kt_rawint4_moe_layer* layer, int32_t tokens, Dims* d) {
  const int rc = check_layer_dims(layer, tokens, d, true);
  if (rc) return rc;
  if (tokens > KT_MOE_DECODE_MAX_TOKENS || d->Ms > KT_MOE_DECODE_MAX_SLOTS)
    return set_error(KT_RAWINT4_EINVAL, "at most 64 tokens and 1024 token-slots: use kt_rawint4_moe_infer");
  return KT_RAWINT4_OK;
}

template <bool MX, bool LORA>
static void launch_decode(const DecodeArgs& a, hipStream_t st) {
  if (LORA) {
    k_decode_lora_a<false><<<dim3((unsigned)((2 * a.R + 3) / 4), (unsigned)a.S), 256, 0, st>>>(a);
    note_launch();
  }
  k_decode_gate_up<MX, LORA><<<dim3((unsigned)(a.I / 16), (unsigned)a.S), 256, 0, st>>>(a);
  note_launch();
  if (LORA) {
    k_decode_lora_a<true><<<dim3((unsigned)((a.R + 3) / 4), (unsigned)a.S), 256, 0, st>>>(a);
    note_launch();
  }
  k_decode_down<MX, LORA><<<(unsigned)(a.H / 16), 512, (size_t)kDownWaves * a.T * 64, st>>>(a);
  note_launch();
}

}  // namespace kt

using namespace kt;

extern "C" {

size_t kt_moe_decode_workspace_bytes(const kt_rawint4_moe_layer* layer, int32_t tokens) {
  Dims d;
  if (check_decode(layer, tokens, &d)) return 0;
  set_error(KT_RAWINT4_OK, "");
  return plan_decode(d).total;
}

int kt_moe_decode(const kt_rawint4_moe_layer* layer, int32_t tokens, const uint16_t* inputs, const int64_t* expert_ids,
                  const float* route_weights, uint16_t* output, void* workspace, size_t workspace_bytes,
                  void* stream) {
  Dims d;
  int rc = check_decode(layer, tokens, &d);
  if (rc) return rc;
  if (tokens == 0) return set_error(KT_RAWINT4_OK, "");
  if (!inputs || !expert_ids || !route_weights || !output)
    return set_error(KT_RAWINT4_EINVAL, "inputs, expert_ids, route_weights and output must be non-NULL");
  if (!is_aligned(inputs, 16) || !is_aligned(output, 2) || !is_aligned(expert_ids, 8) || !is_aligned(route_weights, 4))
    return set_error(KT_RAWINT4_EINVAL, "inputs must be 16-byte aligned, expert_ids 8-byte, the rest by their type");
  const DecodePlan p = plan_decode(d);
  rc = check_caller_workspace(workspace, workspace_bytes, p.total);
  if (rc) return rc;
  DecodeArgs a{};
  a.S = (int)d.Ms, a.k = (int)d.K, a.T = tokens;
  a.E = (int)d.E, a.H = (int)d.H, a.I = (int)d.I, a.R = (int)d.R;
  a.sc = d.sc;
  a.limit = d.limit;
  a.x = inputs;
  a.ids = expert_ids;
  a.rw = route_weights;
  a.out = output;
  a.wg = layer->gate_packed, a.wu = layer->up_packed, a.wd = layer->down_packed;
  a.sg = layer->gate_scale, a.su = layer->up_scale, a.sd = layer->down_scale;
  a.ag = layer->gate_lora_a, a.bg = layer->gate_lora_b, a.au = layer->up_lora_a, a.bu = layer->up_lora_b;
  a.ad = layer->down_lora_a, a.bd = layer->down_lora_b;
  a.h = ws_ptr<float>(workspace, p.h);
  a.hs = ws_ptr<uint16_t>(workspace, p.hs);
  a.next = ws_ptr<int32_t>(workspace, p.next);
  a.lead = ws_ptr<int32_t>(workspace, p.lead);
  a.ua = ws_ptr<float>(workspace, p.ua);
  a.ud = ws_ptr<float>(workspace, p.ud);
  hipStream_t st = static_cast<hipStream_t>(stream);
  begin_launches();
  if (d.fmt == KT_RAWINT4_FORMAT_MXFP4)
    d.R ? launch_decode<true, true>(a, st) : launch_decode<true, false>(a, st);
  else
    d.R ? launch_decode<false, true>(a, st) : launch_decode<false, false>(a, st);
  return finish_launches();
}

}  // extern "C"
