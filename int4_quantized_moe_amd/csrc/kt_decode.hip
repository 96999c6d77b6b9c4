// The routed experts for a few tokens (decoding): gate and up in one kernel,
// down with the weighted sum over the slots in another, two small ones more with LoRA.
//
// With few tokens an expert has one or two of them, and the time is that of
// reading its packed rows once.  So the loads decide the layout: eight lanes
// take 128 bytes of a row in a row, eight rows a load, and a lane's 16 bytes are
// one scale group, which it multiplies by itself:
//   RAWINT4: a code c becomes 1 + c / 16, by a shift and an and-or for two of
//   them, exact in bf16, and
//     sum (c - 8) x = 16 (sum (1 + c / 16) x - 3/2 sum x)
//   by dot products of two with fp32 sums that start from -3/2 sum x of the group.
//   MXFP4: a code is converted to bf16 as it is, the sum starts from 0.
// The scale then multiplies the group's sum in fp32.  Products are exact,
// whatever the inputs' and scales' size.  Inputs are bf16 as given; h, fp32,
// enters as two bf16 (hi and lo), 2^-16 of it left out.
//
// (The MFMAs' operand layout has another row in every lane of 16: their loads
// touch 16 lines where these touch 2, which is what bounded them, 3.4 TB/s.)
#include "kt_step_common.hpp"

#include <math.h>

#include <type_traits>

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
  float* hsum;    // [S][I / 16]: sums of 16 values of h
  int32_t* next;  // [S]: the next slot of the same expert, -1 for none
  int32_t* lead;  // [S]: whether the slot is its expert's first
  float* ua;      // [S][2 R]: x A_g^T | x A_u^T
  float* ud;      // [S][R]: h A_d^T
};

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
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a), __builtin_bit_cast(bf16x2_t, b), c, false);
}

// Loads through a buffer descriptor: a base and an offset that are the same in
// all lanes, and the lane's 32-bit offset.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00020000);
}

// One expert's matrix of so many rows, G scale groups each.
struct Matrix {
  Buffer w, s;
};
__device__ __forceinline__ Matrix matrix_of(const uint8_t* w, const uint16_t* s, size_t e, int rows, int G) {
  const size_t n = (size_t)rows * G;
  return {buffer_of(w + e * n * 16, n * 16), buffer_of(s + e * n, n * 2)};
}

// A contraction goes in units of 256 values, 8 groups, one for each of a row's
// eight lanes.  Codes and scale of this lane's group in rows r .. r + 7 (a tile).
// Every load is issued, whatever the unit, so that how many are in flight
// behind a value is known where it is waited for; a lane whose group lies behind the
// row's last reads that one, and its vectors are 0.
struct Codes {
  u32x4 c;
  uint16_t s;
};
__device__ __forceinline__ void load_codes(const Matrix& m, uint32_t group, uint32_t base, Codes& c) {
  c.c = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(m.w, (int)(group * 16), (int)(base * 16), 0));
  c.s = __builtin_amdgcn_raw_buffer_load_b16(m.s, (int)(group * 2), (int)(base * 2), 0);
}

// Vectors in LDS: four planes of 16 bytes a group, so that eight lanes read 128 bytes in a row.
struct Vec {
  u32x4 v[4];
};
__device__ __forceinline__ void read_vec(const uint8_t* p, int group, int plane, Vec& v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v.v[j] = *reinterpret_cast<const u32x4*>(p + j * plane + group * 16);
}

// The group's product with V vectors, from the sums t[] on.
template <bool MX, int V>
__device__ __forceinline__ void multiply(const u32x4& c, const Vec* x, float* t) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4 w = codes_bf16<MX>(c[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) t[v] = dot2(w[i], x[v].v[j][i], t[v]);
  }
}

// A sum over the eight lanes of a row, in all of them.
__device__ __forceinline__ float eight_sum(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  return v + dpp_f<0x141>(v);
}

constexpr int kLoraParts = 8;  // runs of the ranks
constexpr int kUpDepth = 2;    // units of loads ahead, gate and up

// Gate and up.  A workgroup has 16 columns of I of one expert (its first
// slot's block; the others leave at once) for all of its tokens, V at a time,
// which lie in LDS.  Its four waves split the contraction.
template <bool MX, bool LORA, int V>
__global__ __launch_bounds__(256, 4) void k_decode_gate_up(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t list[KT_MOE_DECODE_MAX_SLOTS];
  __shared__ float red[2][4][V][16];
  __shared__ float lora[LORA ? kLoraParts : 1][2][V][16];
  const int slot = blockIdx.y, i0 = blockIdx.x * 16;
  const int kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t e = a.ids[slot];
  int next = -1, M = 0;
  if (e >= 0 && e < a.E) M = slots_of(a, slot, e, list, next);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.next[slot] = next;
    a.lead[slot] = M > 0;
  }
  if (!M) return;
  const int G = a.H / 32, units = (G + 7) / 8, per = (units + 3) / 4, u0 = kw * per;
  const int Gp = per * 32, plane = Gp * 16;      // groups and bytes of a plane in LDS, 0 behind the row's end
  float* sums = reinterpret_cast<float*>(lds + V * 4 * plane);  // [vectors][Gp]: -3/2 of a group's sum
  const Matrix mg = matrix_of(a.wg, a.sg, e, a.I, G), mu = matrix_of(a.wu, a.su, e, a.I, G);
  const int c8 = lane & 7, row = lane >> 3;
  const uint32_t first = (uint32_t)(i0 + row) * G, rows8 = 8u * G;
  __syncthreads();
  for (int m0 = 0; m0 < M; m0 += V) {
    const int nt = min(V, M - m0);
    Codes cd[kUpDepth][4];  // gate rows 0..7, 8..15, up rows 0..7, 8..15
    auto load = [&](int u, int b) {
      const uint32_t g = first + min(8 * u + c8, G - 1);
      load_codes(mg, g, 0, cd[b][0]);
      load_codes(mg, g, rows8, cd[b][1]);
      load_codes(mu, g, 0, cd[b][2]);
      load_codes(mu, g, rows8, cd[b][3]);
      __builtin_amdgcn_sched_barrier(0);  // (units' loads stay in order)
    };
#pragma unroll
    for (int b = 0; b < kUpDepth; ++b) load(u0 + b, b);
    for (int p = 0; p < nt; ++p) {
      const uint16_t* x = a.x + (size_t)(list[m0 + p] / a.k) * a.H;
      for (int c = threadIdx.x; c < Gp * 4; c += 256) {
        u32x4 v = {0, 0, 0, 0};
        if (c < G * 4) v = *reinterpret_cast<const u32x4*>(x + c * 8);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s += bf_lo(v[j]) + bf_hi(v[j]);
        s += dpp_f<0xB1>(s);
        s += dpp_f<0x4E>(s);
        *reinterpret_cast<u32x4*>(lds + (p * 4 + (c & 3)) * plane + (c >> 2) * 16) = MX ? v : order8(v);
        if ((c & 3) == 0) sums[p * Gp + (c >> 2)] = MX ? 0.f : -1.5f * s;
      }
    }
    if (LORA) {
      // columns by gate and up by runs of the ranks
      const int c = threadIdx.x & 15, up = threadIdx.x >> 4 & 1, part = threadIdx.x >> 5;
      const int len = (a.R + kLoraParts - 1) / kLoraParts, r0 = part * len, r1 = min(a.R, r0 + len);
      const float* b = (up ? a.bu : a.bg) + ((size_t)e * a.I + i0 + c) * a.R;
      float t[V] = {};
#pragma unroll 1
      for (int r = r0; r < r1; ++r) {
        const float w = b[r];
#pragma unroll
        for (int p = 0; p < V; ++p)
          if (p < nt) t[p] = fmaf(w, a.ua[(size_t)list[m0 + p] * 2 * a.R + up * a.R + r], t[p]);
      }
#pragma unroll
      for (int p = 0; p < V; ++p) lora[part][up][p][c] = t[p];
    }
    __syncthreads();
    float acc[4][V] = {};
    for (int v = 0; v < per; v += kUpDepth) {
#pragma unroll
      for (int b = 0; b < kUpDepth; ++b) {
        if (v + b < per) {
          const int g = 8 * (u0 + v + b) + c8;
          Vec x[V];
          float sum[V];
#pragma unroll
          for (int p = 0; p < V; ++p) {
            read_vec(lds + p * 4 * plane, g, plane, x[p]);
            sum[p] = sums[p * Gp + g];
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            float d[V];
#pragma unroll
            for (int p = 0; p < V; ++p) d[p] = sum[p];
            multiply<MX, V>(cd[b][t].c, x, d);
#pragma unroll
            for (int p = 0; p < V; ++p) acc[t][p] = fmaf(bf16_to_float(cd[b][t].s), d[p], acc[t][p]);
            __builtin_amdgcn_sched_barrier(0);  // (decoded tiles side by side take registers from the loads ahead)
          }
        }
        load(u0 + v + b + kUpDepth, b);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int p = 0; p < V; ++p) {
        const float v = eight_sum(acc[t][p]);
        if (c8 == 0) red[t >> 1][kw][p][(t & 1) * 8 + row] = v;
      }
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
      const float sum = row16_sum(bf16_to_float(hi) + bf16_to_float(lo));
      if (c == 0) a.hsum[(size_t)s * (a.I / 16) + blockIdx.x] = sum;
      if (LORA) a.h[(size_t)s * a.I + i0 + c] = h;
    }
    if (m0 + V < M) __syncthreads();
  }
}

constexpr int kVecs = 4;  // tokens that a row of A takes at a time
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


constexpr int kDownWaves = 4;
constexpr int kDownDepth = 4;  // units of loads ahead
constexpr int kDownK = 64;     // groups of h in LDS at a time

// Down and the sum over the slots.  A workgroup has 16 columns of H; its waves
// take the experts in turn (a wave per expert, the whole contraction), a slot at a
// time with its h in LDS, and add to sums of their own per token, which the end
// joins in the waves' order.
template <bool MX, bool LORA>
__global__ __launch_bounds__(64 * kDownWaves, 4) void k_decode_down(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t order[KT_MOE_DECODE_MAX_SLOTS], expert[KT_MOE_DECODE_MAX_SLOTS];
  __shared__ int16_t next[KT_MOE_DECODE_MAX_SLOTS];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c8 = lane & 7, row = lane >> 3;
  const int h0 = blockIdx.x * 16, G = a.I / 32;
  constexpr int plane = kDownK * 16;
  uint8_t* hl = lds + wave * (8 * plane + kDownK * 4);  // hi's four planes, lo's four, -3/2 of the groups' sums
  float* sums = reinterpret_cast<float*>(hl + 8 * plane);
  float* acc = reinterpret_cast<float*>(lds + kDownWaves * (8 * plane + kDownK * 4));  // [waves][T][16]
  int U = 0;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const int s = s0 + lane;
    const bool lead = s < a.S && a.lead[s];
    const uint64_t mask = __ballot(lead);
    if (wave == 0) {
      if (s < a.S) next[s] = (int16_t)a.next[s];
      if (lead) {
        const int at = U + __popcll(mask & ((1ull << lane) - 1));
        order[at] = (uint16_t)s;
        expert[at] = (uint16_t)a.ids[s];
      }
    }
    U += __popcll(mask);
  }
  for (int i = threadIdx.x; i < kDownWaves * a.T * 16; i += 64 * kDownWaves) acc[i] = 0.f;
  __syncthreads();
  const uint32_t first = (uint32_t)(h0 + row) * G, rows8 = 8u * G;
  for (int j = wave; j < U; j += kDownWaves) {
    const size_t e = __builtin_amdgcn_readfirstlane(expert[j]);
    const Matrix md = matrix_of(a.wd, a.sd, e, a.H, G);
    for (int s = __builtin_amdgcn_readfirstlane(order[j]); s >= 0; s = __builtin_amdgcn_readfirstlane(next[s])) {
      float y[2] = {0.f, 0.f};
      for (int k0 = 0; k0 < G; k0 += kDownK) {
        const int len = min(kDownK, G - k0), units = (len + 7) / 8;
        Codes cd[kDownDepth][2];
        auto load = [&](int u, int b) {
          const uint32_t g = first + min(k0 + 8 * u + c8, G - 1);
          load_codes(md, g, 0, cd[b][0]);
          load_codes(md, g, rows8, cd[b][1]);
          __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int b = 0; b < kDownDepth; ++b) load(b, b);
        wave_fence();
        // (16 bytes of hi or lo: a quarter of a group)
        for (int c = lane; c < units * 32; c += 64) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            u32x4 v = {0, 0, 0, 0};
            if (c < len * 4) v = *reinterpret_cast<const u32x4*>(a.hs + ((size_t)s * 2 + p) * a.I + k0 * 32 + c * 8);
            *reinterpret_cast<u32x4*>(hl + (p * 4 + (c & 3)) * plane + (c >> 2) * 16) = v;
          }
        }
        if (lane < units * 8) {
          float t = 0.f;
          if (!MX && lane < len) {
            const float* p = a.hsum + (size_t)s * (a.I / 16) + (k0 + lane) * 2;
            t = -1.5f * (p[0] + p[1]);
          }
          sums[lane] = t;
        }
        wave_fence();
        for (int u = 0; u < units; u += kDownDepth) {
#pragma unroll
          for (int b = 0; b < kDownDepth; ++b) {
            if (u + b < units) {
              const int g = 8 * (u + b) + c8;
              Vec x[2];
              read_vec(hl, g, plane, x[0]);
              read_vec(hl + 4 * plane, g, plane, x[1]);
              const float sum = sums[g];
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                float d[2] = {sum, 0.f};
                multiply<MX, 2>(cd[b][t].c, x, d);
                y[t] = fmaf(bf16_to_float(cd[b][t].s), d[0] + d[1], y[t]);
              }
            }
            load(u + b + kDownDepth, b);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        y[t] = eight_sum(y[t]);
        if (!MX) y[t] *= 16.f;
        if (LORA) {
          // an eighth of the ranks a lane
          const float *b = a.bd + (e * a.H + h0 + 8 * t + row) * a.R, *u = a.ud + (size_t)s * a.R;
          float l = 0.f;
#pragma unroll 1
          for (int r = c8; r < a.R; r += 8) l = fmaf(b[r], u[r], l);
          y[t] = fmaf(a.sc, eight_sum(l), y[t]);
        }
      }
      if (c8 == 0) {
        float* o = acc + (wave * a.T + s / a.k) * 16 + row;
        o[0] = fmaf(a.rw[s], y[0], o[0]);
        o[8] = fmaf(a.rw[s], y[1], o[8]);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += 64 * kDownWaves) {
    float v = 0.f;
    for (int w = 0; w < kDownWaves; ++w) v += acc[w * a.T * 16 + i];
    a.out[(size_t)(i >> 4) * a.H + h0 + (i & 15)] = float_to_bf16(v);
  }
}

// ---------------------------------------------------------------- host

struct DecodePlan {
  size_t hs, hsum, h, next, lead, ua, ud, total;
};
static DecodePlan plan_decode(const Dims& d) {
  DecodePlan p;
  const size_t S = (size_t)d.Ms;
  p.next = 0;
  p.lead = round256(4 * S);
  p.hs = p.lead + round256(4 * S);
  p.hsum = p.hs + round256(4 * S * d.I);
  p.h = p.hsum + round256(4 * S * (d.I / 16));
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
  const size_t groups = (size_t)((a.H / 32 + 7) / 8 + 3) / 4 * 32;
  const dim3 grid((unsigned)(a.I / 16), (unsigned)a.S);
  if (a.T == 1)
    k_decode_gate_up<MX, LORA, 1><<<grid, 256, groups * 68, st>>>(a);
  else
    k_decode_gate_up<MX, LORA, 2><<<grid, 256, 2 * groups * 68, st>>>(a);
  note_launch();
  if (LORA) {
    k_decode_lora_a<true><<<dim3((unsigned)((a.R + 3) / 4), (unsigned)a.S), 256, 0, st>>>(a);
    note_launch();
  }
  k_decode_down<MX, LORA><<<(unsigned)(a.H / 16), 64 * kDownWaves, kDownWaves * (kDownK * 132 + (size_t)a.T * 64), st>>>(a);
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
  a.hsum = ws_ptr<float>(workspace, p.hsum);
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
