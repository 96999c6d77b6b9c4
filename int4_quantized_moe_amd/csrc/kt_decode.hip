// The routed experts for a few tokens (decoding): gate and up in one kernel,
// down with the weighted sum over the slots in another, two small ones more with LoRA.
//
// With few tokens an expert has one or two of them, and the time is that of
// reading its packed rows once.  Weights go into the MFMAs as bf16, tokens as
// the other operand's rows, one MFMA (32 contraction values) per 16 weight rows and
// scale group, so that the scale multiplies the group's sum in fp32.
//   RAWINT4: a code c becomes 1 + c / 16, by a shift and an and-or for two of
//   them, exact in bf16, and
//     sum (c - 8) x = 16 (sum (1 + c / 16) x - 3/2 sum x),
//   where -3/2 sum x of the group is the MFMA's initial sum.  Products are
//   exact, whatever the inputs' and scales' size.
//   MXFP4: a code is converted to bf16 as it is, the initial sum is 0.
// Inputs are bf16 as given; h, fp32, enters as two bf16 (hi and lo) in two
// rows of the same MFMA, 2^-16 of it left out.
//
// A lane loads 16 bytes of a row, a whole scale group; an exchange of 4 x 4
// dwords between the wave's four rows of 16 lanes gives each MFMA one group.
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
  float* h;       // [S][I]
  int32_t* next;  // [S]: the next slot of the same expert, -1 for none
  int32_t* lead;  // [S]: whether the slot is its expert's first
  float* ua;      // [S][2 R]: x A_g^T | x A_u^T
  float* ud;      // [S][R]: h A_d^T
};

typedef u32x4 u32x4_u2 __attribute__((aligned(2)));

// The slots of slot `s`'s expert from s on, in order, to list[] (wave-uniform
// count); 0 if the slot is dropped or not its expert's first.  Every wave
// finds the same; wave 0 writes.  `next`: the slot after s, or -1.
__device__ __forceinline__ int slots_of(const DecodeArgs& a, int s, uint16_t* list, int& next) {
  const int lane = threadIdx.x & 63;
  const int64_t e = a.ids[s];
  next = -1;
  if (e < 0 || e >= a.E) return 0;
  int n = 0;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const bool hit = s0 + lane < a.S && a.ids[s0 + lane] == e;
    const uint64_t mask = __ballot(hit);
    if (s0 <= s) {
      // a hit before s: another slot leads
      const uint64_t before = s - s0 >= 64 ? ~0ull : (1ull << (s - s0)) - 1;
      if (mask & before) n = -1024 * 1024;
    }
    const int at = n + __popcll(mask & ((1ull << lane) - 1));
    if (hit && at >= 0 && threadIdx.x < 64) list[at] = (uint16_t)(s0 + lane);
    if (next < 0) {
      uint64_t after = mask;
      if (s0 + 63 <= s) after = 0;
      else if (s0 <= s) after &= ~((2ull << (s - s0)) - 1);
      if (after) next = s0 + __ffsll((unsigned long long)after) - 1;
    }
    n += __popcll(mask);
  }
  return n > 0 ? n : 0;
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

// 16 weight rows from `w` (row pitch K / 2 bytes) and `sc` (pitch K / 32), contraction
// groups 4 it .. 4 it + 3: codes and scales of this lane's row.
struct RowTile {
  const uint8_t* w;
  const uint16_t* s;
  int G;  // groups of a row
};
__device__ __forceinline__ u32x4 tile_codes(const RowTile& t, int it, int q) {
  return 4 * it + q < t.G ? *reinterpret_cast<const u32x4*>(t.w + (size_t)(4 * it + q) * 16) : u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ void tile_scales(const RowTile& t, int it, float* s) {
#pragma unroll
  for (int g = 0; g < 4; ++g) s[g] = 4 * it + g < t.G ? bf16_to_float(t.s[4 * it + g]) : 0.f;
}

constexpr int kPadRow = 16;  // bytes between the rows of LDS planes, beyond their length

// Gate and up.  A workgroup has 16 columns of I of one expert (its first
// slot's block; the others leave at once) for all of its tokens, P at a time;
// the four waves split the contraction.  Lane l: weight row l % 16, MFMA row 4 (l / 16) is token l / 16 (of P = 4).
template <bool MX, int P>
__global__ __launch_bounds__(256) void k_decode_gate_up(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t list[KT_MOE_DECODE_MAX_SLOTS];
  __shared__ float red[4][2][4][16];
  const int slot = blockIdx.y, i0 = blockIdx.x * 16;
  int next;
  const int M = slots_of(a, slot, list, next);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.next[slot] = next;
    a.lead[slot] = M > 0;
  }
  if (!M) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t e = a.ids[slot];
  const int G = a.H / 32, its = (G + 3) / 4, pitch = its * 256 + kPadRow, gp = its * 4;
  uint8_t* xs = lds;                                          // [P][pitch]: tokens in the codes' order
  float* sum = reinterpret_cast<float*>(lds + P * pitch);     // [P][gp]: -3/2 of a group's sum
  const size_t row = (size_t)e * a.I + i0 + n;
  const RowTile tg{a.wg + row * (a.H / 2), a.sg + row * G, G}, tu{a.wu + row * (a.H / 2), a.su + row * G, G};
  const int tok = P == 4 ? q : P == 2 ? q >> 1 : 0;   // whose sums this lane holds
  const int arow = P == 4 ? n >> 2 : P == 2 ? n >> 3 : 0;  // which token's values it hands in
  __syncthreads();
  for (int m0 = 0; m0 < M; m0 += P) {
    const int nt = min(P, M - m0);
    if (m0) __syncthreads();
    for (int p = 0; p < nt; ++p) {
      const uint16_t* x = a.x + (size_t)(list[m0 + p] / a.k) * a.H;
      for (int c = threadIdx.x; c < its * 16; c += 256) {
        u32x4 v = {0, 0, 0, 0};
        if (c * 8 < a.H) v = *reinterpret_cast<const u32x4*>(x + c * 8);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s += bf_lo(v[j]) + bf_hi(v[j]);
        s += dpp_f<0xB1>(s);
        s += dpp_f<0x4E>(s);
        *reinterpret_cast<u32x4*>(xs + p * pitch + c * 16) = MX ? v : order8(v);
        if ((c & 3) == 0) sum[p * gp + (c >> 2)] = MX ? 0.f : -1.5f * s;
      }
    }
    __syncthreads();
    float g = 0.f, u = 0.f;
    const int trow = min(arow, nt - 1), ttok = min(tok, nt - 1);
    for (int it = wave; it < its; it += 4) {
      u32x4 cg = tile_codes(tg, it, q), cu = tile_codes(tu, it, q);
      float sg[4], su[4];
      tile_scales(tg, it, sg);
      tile_scales(tu, it, su);
      uint32_t rg[4] = {cg.x, cg.y, cg.z, cg.w}, ru[4] = {cu.x, cu.y, cu.z, cu.w};
      transpose4(rg);
      transpose4(ru);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 xv = *reinterpret_cast<const u32x4*>(xs + trow * pitch + it * 256 + j * 64 + q * 16);
        const float c0 = sum[ttok * gp + it * 4 + j];
        const floatx4 init = {c0, 0.f, 0.f, 0.f};
        g = fmaf(sg[j], mfma_bf16(xv, codes_bf16<MX>(rg[j]), init).x, g);
        u = fmaf(su[j], mfma_bf16(xv, codes_bf16<MX>(ru[j]), init).x, u);
      }
    }
    // (P < 4: rows of lanes that hold the same token hold the same sums)
    red[wave][0][q][n] = g;
    red[wave][1][q][n] = u;
    __syncthreads();
    if (threadIdx.x < 16 * nt) {
      const int p = threadIdx.x >> 4, c = threadIdx.x & 15, qr = P == 4 ? p : P == 2 ? 2 * p : 0;
      const float by = MX ? 1.f : 16.f;
      float gv = 0.f, uv = 0.f;
      for (int w = 0; w < 4; ++w) gv += red[w][0][qr][c], uv += red[w][1][qr][c];
      gv *= by, uv *= by;
      const int s = list[m0 + p];
      if (a.R) {
        const float *bg = a.bg + ((size_t)e * a.I + i0 + c) * a.R, *bu = a.bu + ((size_t)e * a.I + i0 + c) * a.R;
        const float *ug = a.ua + (size_t)s * 2 * a.R, *uu = ug + a.R;
        float lg = 0.f, lu = 0.f;
        for (int r = 0; r < a.R; ++r) lg = fmaf(bg[r], ug[r], lg), lu = fmaf(bu[r], uu[r], lu);
        gv = fmaf(a.sc, lg, gv), uv = fmaf(a.sc, lu, uv);
      }
      if (a.limit > 0.f) {
        // (comparisons that keep a NaN)
        gv = gv > a.limit ? a.limit : gv;
        uv = uv > a.limit ? a.limit : uv < -a.limit ? -a.limit : uv;
      }
      a.h[(size_t)s * a.I + i0 + c] = gv * sigmoid_f(gv) * uv;
    }
  }
}

// x A_g^T | x A_u^T of every slot (DOWN: h A_d^T): a wave per row of A of an expert, for all of its tokens.
template <bool DOWN>
__global__ __launch_bounds__(256) void k_decode_lora_a(DecodeArgs a) {
  __shared__ uint16_t list[KT_MOE_DECODE_MAX_SLOTS];
  int next;
  const int M = slots_of(a, blockIdx.y, list, next);
  if (!M) return;
  __syncthreads();
  const int rows = DOWN ? a.R : 2 * a.R, r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (r >= rows) return;
  const size_t e = (size_t)a.ids[blockIdx.y];
  const int K = DOWN ? a.I : a.H;
  const float* w = (DOWN ? a.ad : r < a.R ? a.ag : a.au) + (e * a.R + (r < a.R ? r : r - a.R)) * K;
  for (int m = 0; m < M; ++m) {
    const int s = list[m];
    float v = 0.f;
    for (int c = lane * 4; c < K; c += 256) {
      const float4 b = *reinterpret_cast<const float4*>(w + c);
      float4 x;
      if (DOWN) {
        x = *reinterpret_cast<const float4*>(a.h + (size_t)s * K + c);
      } else {
        const u32pair p = *reinterpret_cast<const u32pair*>(a.x + (size_t)(s / a.k) * K + c);
        x = float4{bf_lo(p.x), bf_hi(p.x), bf_lo(p.y), bf_hi(p.y)};
      }
      v = fmaf(b.x, x.x, v);
      v = fmaf(b.y, x.y, v);
      v = fmaf(b.z, x.z, v);
      v = fmaf(b.w, x.w, v);
    }
    v = wave_sum(v);
    if (lane == 0) (DOWN ? a.ud : a.ua)[(size_t)s * rows + r] = v;
  }
}

constexpr int kDownWaves = 8;
constexpr int kDownK = 2048;  // contraction values of h staged at a time

// Down and the sum over the slots.  A workgroup has 16 columns of H; its waves
// take the experts in turn (a wave per expert, the whole contraction) for one token at a time
// and add to sums of their own per token, which the end joins in the waves' order.
template <bool MX>
__global__ __launch_bounds__(512) void k_decode_down(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t order[KT_MOE_DECODE_MAX_SLOTS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int h0 = blockIdx.x * 16;
  const int G = a.I / 32, kc = min(a.I, kDownK), gp = (kc / 32 + 3) / 4 * 4;
  const int plane = gp * 64 + kPadRow;  // bytes of the hi or the lo plane
  const int stage = 2 * plane + gp * 4;
  uint8_t* hs = lds + wave * stage;
  float* sum = reinterpret_cast<float*>(hs + 2 * plane);
  float* acc = reinterpret_cast<float*>(lds + kDownWaves * stage);  // [waves][T][16]
  for (int i = threadIdx.x; i < kDownWaves * a.T * 16; i += 512) acc[i] = 0.f;
  int U = 0;
  for (int s0 = 0; s0 < a.S; s0 += 64) {
    const bool lead = s0 + lane < a.S && a.lead[s0 + lane];
    const uint64_t mask = __ballot(lead);
    if (lead && wave == 0) order[U + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)(s0 + lane);
    U += __popcll(mask);
  }
  __syncthreads();
  for (int j = wave; j < U; j += kDownWaves) {
    const int first = order[j];
    const size_t e = (size_t)a.ids[first], row = e * a.H + h0 + n;
    for (int s = first; s >= 0; s = a.next[s]) {
      float y = 0.f;
      for (int k0 = 0; k0 < a.I; k0 += kDownK) {
        const int len = min(kDownK, a.I - k0), g0 = k0 / 32, g1 = (len / 32 + 3) / 4 * 4;
        wave_fence();
        // 4 values a lane to hi and lo planes; an even lane and its neighbour make 16 bytes of each
        for (int c = lane * 4; c < g1 * 32; c += 256) {
          float4 v = {0, 0, 0, 0};
          if (c < len) v = *reinterpret_cast<const float4*>(a.h + (size_t)s * a.I + k0 + c);
          const float f[4] = {v.x, v.y, v.z, v.w};
          uint16_t hi[4], lo[4];
          float t = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            split_bf16(f[i], hi[i], lo[i]);
            t += bf16_to_float(hi[i]) + bf16_to_float(lo[i]);
          }
          t += dpp_f<0xB1>(t);
          t += dpp_f<0x4E>(t);
          t += dpp_f<0x141>(t);
          const uint32_t h01 = pack2(hi[0], hi[1]), h23 = pack2(hi[2], hi[3]);
          const uint32_t l01 = pack2(lo[0], lo[1]), l23 = pack2(lo[2], lo[3]);
          // even lanes make the hi plane's 16 bytes, odd ones the lo plane's
          const bool odd = lane & 1;
          const uint32_t p01 = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? h01 : l01), 0xB1, 0xf, 0xf, true);
          const uint32_t p23 = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? h23 : l23), 0xB1, 0xf, 0xf, true);
          const u32x4 v8 = odd ? u32x4{p01, p23, l01, l23} : u32x4{h01, h23, p01, p23};
          *reinterpret_cast<u32x4*>(hs + (odd ? plane : 0) + (c >> 3) * 16) = MX ? v8 : order8(v8);
          if ((lane & 7) == 0) sum[c >> 5] = MX ? 0.f : -1.5f * t;
        }
        wave_fence();
        const RowTile t{a.wd + row * (a.I / 2) + k0 / 2, a.sd + row * G + g0, len / 32};
        for (int it = 0; it < g1 / 4; ++it) {
          const u32x4 cd = tile_codes(t, it, q);
          float sd[4];
          tile_scales(t, it, sd);
          uint32_t rd[4] = {cd.x, cd.y, cd.z, cd.w};
          transpose4(rd);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // MFMA rows in turn: hi, lo
            const u32x4 hv = *reinterpret_cast<const u32x4*>(hs + (n & 1) * plane + it * 256 + g * 64 + q * 16);
            const floatx4 d = mfma_bf16(hv, codes_bf16<MX>(rd[g]), floatx4{sum[it * 4 + g], 0.f, 0.f, 0.f});
            y = fmaf(sd[g], d.x + d.y, y);
          }
        }
      }
      if (!MX) y *= 16.f;
      if (a.R) {
        // a quarter of the ranks a row of lanes
        const float *b = a.bd + row * a.R, *u = a.ud + (size_t)s * a.R;
        float t = 0.f;
        for (int r = q; r < a.R; r += 4) t = fmaf(b[r], u[r], t);
        y = fmaf(a.sc, rows_sum(t), y);
      }
      if (q == 0) {
        float* o = acc + (wave * a.T + s / a.k) * 16 + n;
        *o = fmaf(a.rw[s], y, *o);
      }
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
  size_t h, next, lead, ua, ud, total;
};
static DecodePlan plan_decode(const Dims& d) {
  DecodePlan p;
  const size_t S = (size_t)d.Ms;
  p.next = 0;
  p.lead = round256(4 * S);
  p.h = p.lead + round256(4 * S);
  p.ua = p.h + round256(4 * S * d.I);
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

constexpr size_t kLdsMost = 160 * 1024;

static size_t gate_up_lds(int H, int P) {
  const size_t its = (size_t)(H / 32 + 3) / 4;
  return P * (its * 256 + kPadRow) + P * its * 16;
}

template <bool MX>
static void launch_decode(const DecodeArgs& a, hipStream_t st) {
  if (a.R) {
    k_decode_lora_a<false><<<dim3((unsigned)((2 * a.R + 3) / 4), (unsigned)a.S), 256, 0, st>>>(a);
    note_launch();
  }
  int P = a.T >= 4 ? 4 : a.T >= 2 ? 2 : 1;
  while (P > 1 && gate_up_lds(a.H, P) + 8192 > kLdsMost) P /= 2;
  const dim3 grid((unsigned)(a.I / 16), (unsigned)a.S);
  const size_t lds = gate_up_lds(a.H, P);
  if (P == 4)
    k_decode_gate_up<MX, 4><<<grid, 256, lds, st>>>(a);
  else if (P == 2)
    k_decode_gate_up<MX, 2><<<grid, 256, lds, st>>>(a);
  else
    k_decode_gate_up<MX, 1><<<grid, 256, lds, st>>>(a);
  note_launch();
  if (a.R) {
    k_decode_lora_a<true><<<dim3((unsigned)((a.R + 3) / 4), (unsigned)a.S), 256, 0, st>>>(a);
    note_launch();
  }
  const int kc = a.I < kDownK ? a.I : kDownK, gp = (kc / 32 + 3) / 4 * 4;
  const size_t stage = 2 * (gp * 64 + kPadRow) + gp * 4;
  k_decode_down<MX><<<(unsigned)(a.H / 16), 512, kDownWaves * (stage + (size_t)a.T * 64), st>>>(a);
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
  a.next = ws_ptr<int32_t>(workspace, p.next);
  a.lead = ws_ptr<int32_t>(workspace, p.lead);
  a.ua = ws_ptr<float>(workspace, p.ua);
  a.ud = ws_ptr<float>(workspace, p.ud);
  begin_launches();
  if (d.fmt == KT_RAWINT4_FORMAT_MXFP4)
    launch_decode<true>(a, static_cast<hipStream_t>(stream));
  else
    launch_decode<false>(a, static_cast<hipStream_t>(stream));
  return finish_launches();
}

}  // extern "C"
