// The routed experts for a few tokens (decoding): gate and up in one kernel,
// down with the weighted sum over the slots in another, two small ones more with LoRA, and one
// that adds down's parts where it is split.
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
// The scale then multiplies the group's sum in fp32.  Products are exact, subnormal inputs
// and scales among them, and sums stay in fp32's range for inputs up to 2^120
// (3/2 of 32 of them).  Inputs are bf16 as given.  h enters down with
// a power of two for 16 columns: for RAWINT4 as integers of 24 bits, whose three bytes are multiplied
// with the codes by dot products of four, exactly,
//     sum (c - 8) q = 2^16 sum c q2 + 2^8 sum c q1 + sum c q0 - 8 sum q
// (fewer instructions than fp16 takes, and 2^-23 of the largest of the 16), for MXFP4 as the sum of two fp16
// numbers (2^-22 of itself).  One fp16 number would do 2^-11, which shows in outputs that are small differences.
//
// 384 experts, 8 a token, 7168 x 2048: one token 40 us (195 MB of codes and scales: 4.9 TB/s), 4 tokens with LoRA of rank
// 64 196 us, 8 tokens on MXFP4 251 to 258 us (1.4 GB: 5.8 TB/s), 32 tokens with rank 16 and padded slots 888 to 907 us.
// Gate and up read an expert's codes once for two of its slots, down once for every slot (with the
// hint that a second pass is not expected: 32 tokens read 2.0 GB there, of 1.5 GB that are different).
// Passes over codes that mostly lie in the caches are bound by the multiplications: 8 experts, rank 16, of 4 tokens
// 117 us, of 8 215, of 32 797; the batched forward, which is made for that, takes 179, 180 and 202.  Short rows have a kernel of
// their own for gate and up, and down split over the experts: 8 tokens of 279 experts, 576 x 2016, 60 us (floor 29).
//
// (The MFMAs' operand layout has another row in every lane of 16: their loads
// touch 16 lines where these touch 2, which is what bounded them, 3.4 TB/s.)
#include "kt_step_common.hpp"

#include <math.h>

#include <type_traits>

namespace kt {

typedef u32x4 u32x4_u2 __attribute__((aligned(2)));
typedef u32pair u32pair_u2 __attribute__((aligned(2)));

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
  uint8_t* hs;    // [S][I / 1024, upwards][planes][32][16 bytes]: h as down reads it (finish_column)
  float2_t* hsf;  // [S][I / 16]: RAWINT4: -8 times the sum of 16 columns (an int); what their products with the codes are to be multiplied by
  int32_t* next;  // [S]: the next slot of the same expert, -1 for none
  int32_t* lead;  // [S]: whether the slot is its expert's first
  float* ua;      // [S][2 R]: x A_g^T | x A_u^T
  float* ud;      // [S][R]: h A_d^T
  float* part;    // [parts][T][H]: down's sums, where it is split
  int by_slot;    // a workgroup of gate and up takes two slots, a wave of down one, not all of an expert's
};

// The slots of an expert, in order, by the masks of all slots that chose it.
constexpr int kSlotWords = KT_MOE_DECODE_MAX_SLOTS / 64;
struct Slots {
  const uint64_t* mask;  // in LDS
  int word;
  uint64_t rest;
  __device__ __forceinline__ int take() {  // the next slot; there has to be one
    while (!rest) rest = get(++word);
    const int s = word * 64 + __ffsll((unsigned long long)rest) - 1;
    rest &= rest - 1;
    return s;
  }
  __device__ __forceinline__ uint64_t get(int w) const {
    const uint64_t m = mask[w];
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(m >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)m);
  }
};
// A workgroup's slots: those of slot s's expert e, if s is its first (count > 0); next: the one after s, or -1; rank: how many
// are before s.  Ends with a barrier.
__device__ __forceinline__ Slots find_slots(const DecodeArgs& a, int s, int64_t e, uint64_t* mask, int& count, int& next,
                                            int& rank) {
  const int words = (a.S + 63) / 64, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, lane = threadIdx.x & 63;
  for (int w = wave; w < words; w += waves) {
    const int i = w * 64 + lane;
    const uint64_t m = __ballot(i < a.S && a.ids[min(i, a.S - 1)] == e);
    if (lane == 0) mask[w] = m;
  }
  __syncthreads();
  Slots r{mask, 0, 0};
  r.rest = r.get(0);
  next = -1;
  int n = 0;
  rank = 0;
  for (int w = 0; w < words; ++w) {
    uint64_t m = r.get(w);
    n += __popcll(m);
    if (w < s >> 6) {
      rank += __popcll(m);
      continue;
    }
    if (w == s >> 6) {
      rank += __popcll(m & ((1ull << (s & 63)) - 1));
      m &= ~((2ull << (s & 63)) - 1);
    }
    if (m && next < 0) next = w * 64 + __ffsll((unsigned long long)m) - 1;
  }
  count = rank ? 0 : n;
  return r;
}

// 8 codes of a dword as two-byte floats: RAWINT4 1 + c / 16 in bf16, in the order k0 k4 k1 k5 k2 k6 k3 k7,
// MXFP4 their values in order, in bf16 or fp16 (HALF).
struct DotConsts {
  uint32_t m, o;
};
__device__ __forceinline__ DotConsts dot_consts() {
  // (values the compiler cannot see through, in a scalar and a vector register: (w & m) | o is then one instruction)
  uint32_t m = 0x00780078u, o = 0x3f803f80u;
  asm volatile("" : "+s"(m));
  asm volatile("" : "+v"(o));
  return DotConsts{m, o};
}
template <bool HALF>
__device__ __forceinline__ u32x4 decode8_mx(uint32_t w) {
  auto two = [&](auto sel) {
    constexpr int k = decltype(sel)::value;
    if (HALF) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, k));
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, k));
  };
  return u32x4{two(std::integral_constant<int, 0>()), two(std::integral_constant<int, 1>()),
               two(std::integral_constant<int, 2>()), two(std::integral_constant<int, 3>())};
}
template <bool MX>
__device__ __forceinline__ u32x4 decode8(uint32_t w, DotConsts dc) {
  if (MX) return decode8_mx<false>(w);
  return u32x4{((w << 3) & dc.m) | dc.o, ((w >> 1) & dc.m) | dc.o, ((w >> 5) & dc.m) | dc.o, ((w >> 9) & dc.m) | dc.o};
}

// 8 two-byte values in order -> the order of RAWINT4's decode8
__device__ __forceinline__ u32x4 order8(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
               __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
template <bool HALF>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  if (HALF) return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2_t, a), __builtin_bit_cast(half2_t, b), c, false);
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a), __builtin_bit_cast(bf16x2_t, b), c, false);
}

// Loads through a buffer descriptor: a base and an offset that are the same in
// all lanes, and the lane's 32-bit offset.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00020000);
}
// kCodes: read once, so that the L2 lets them go first and keeps vectors and scales (one token 43.0 -> 39.8 us, eight on
// MXFP4 255 -> 238).
constexpr int kCodes = 2, kKept = 0;
template <int HOW>
__device__ __forceinline__ u32x4 buffer16(Buffer b, uint32_t lane, uint32_t base) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane, (int)base, HOW));
}

// A contraction goes in units of 256 values, 8 groups, one for each of a row's
// eight lanes; a load brings a unit of eight rows (a tile).  Every load of
// codes is issued, whatever the unit, so that how many are in flight behind a value
// is known where it is waited for: behind the wave's last unit all lanes read the same
// bytes.  A lane whose group lies behind the row's last reads that one, and its
// vectors are 0.

// Vectors in LDS: four planes of 16 bytes a group, so that eight lanes read 128 bytes in a row.
struct Vec {
  u32x4 v[4];
};
__device__ __forceinline__ void read_vec(const uint8_t* p, int group, int plane, Vec& v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v.v[j] = *reinterpret_cast<const u32x4*>(p + j * plane + group * 16);
}

// A sum over the eight lanes of a row, in all of them.
__device__ __forceinline__ float eight_sum(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  return v + dpp_f<0x141>(v);
}

constexpr int kLoraParts = 8;  // runs of the ranks
constexpr int kUpDepth = 2;    // units of loads ahead, gate and up
constexpr int kUpVecs = 2;     // tokens that gate and up take at a time

// What a gate and up workgroup keeps in LDS.
struct UpLds {
  uint8_t* x;        // [V][4][Gp][16 bytes]
  float* sums;       // [V][Gp]: -3/2 of a group's sum
  uint16_t* scales;  // [2][16][G]: of gate and of up
  float* b;          // [2][16][R]: rows of B
  float* ua;         // [V][2 R]
  float (*red)[4][kUpVecs][16];            // [gate, up][wave][token][column]
  float (*lora)[2][kUpVecs][16];           // [run of ranks][gate, up][token][column]
};

constexpr int kStage = 4;  // 16-byte pieces a thread takes at a time while LDS is filled

// (`first`: the thread's first piece)  Pieces of two runs of n, one behind the other in LDS, kStage of a thread's: loads (those behind the end: the
// last piece again) and stores.
template <typename T>
__device__ __forceinline__ void stage_load(const void* p, const void* q, int n, int first, u32x4* v) {
#pragma unroll
  for (int i = 0; i < kStage; ++i) {
    const int c = min(first + 256 * i, 2 * n - 1);
    v[i] = c < n ? *(reinterpret_cast<const T*>(p) + c) : *(reinterpret_cast<const T*>(q) + (c - n));
  }
}
__device__ __forceinline__ void stage_store(void* p, int n, int first, const u32x4* v) {
#pragma unroll
  for (int i = 0; i < kStage; ++i) {
    const int c = first + 256 * i;
    if (c < 2 * n) reinterpret_cast<u32x4*>(p)[c] = v[i];
  }
}
__device__ __forceinline__ void token_load(const uint16_t* x, int n, int first, u32x4* v) {
#pragma unroll
  for (int i = 0; i < kStage; ++i)
    v[i] = *(reinterpret_cast<const u32x4*>(x) + min(first + 256 * i, n - 1));
}
// a token's pieces to its planes, 0 behind the row's end, with the groups' sums
template <bool MX>
__device__ __forceinline__ void stage_token(uint8_t* x, float* sums, int G, int Gp, int first, const u32x4* v) {
#pragma unroll
  for (int i = 0; i < kStage; ++i) {
    const int c = first + 256 * i;
    u32x4 w = v[i];
    if (c >= G * 4) w = u32x4{0, 0, 0, 0};
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) s += bf_lo(w[j]) + bf_hi(w[j]);
    s += dpp_f<0xB1>(s);
    s += dpp_f<0x4E>(s);
    if (c < Gp * 4) {
      *reinterpret_cast<u32x4*>(x + ((c & 3) * Gp + (c >> 2)) * 16) = MX ? w : order8(w);
      if ((c & 3) == 0) sums[c >> 2] = MX ? 0.f : -1.5f * s;
    }
  }
}

// One pass of a workgroup's four waves over its columns for V tokens (slots sl[]): sums to l.red and l.lora.
template <bool MX, bool LORA, int V>
__device__ __forceinline__ void gate_up_pass(const DecodeArgs& a, int64_t e, int i0, const int* sl, bool first_pass,
                                             const UpLds& l) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // (or the addresses below are kept in registers over the passes, which there are too few for)
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c8 = lane & 7, row = lane >> 3;
  const int G = a.H / 32, units = (G + 7) / 8, per = (units + 3) / 4, u0 = kw * per, u1 = min(units, u0 + per);
  const int Gp = per * 32, plane = Gp * 16;  // groups and bytes of a plane in LDS, 0 behind the row's end
  const size_t n = (size_t)a.I * G;
  const Buffer wg = buffer_of(a.wg + e * n * 16, n * 16), wu = buffer_of(a.wu + e * n * 16, n * 16);
  const uint32_t at = (uint32_t)(i0 + row) * G, rows8 = 128u * G;
  // Into LDS: the rows' scales as they lie, 32 G bytes of each matrix, the tokens, and with LoRA rows of B and ua.
  // Their loads are on their way before the first codes', so that waiting for them waits for no codes.
  const uint16_t *sg = a.sg + e * n + (size_t)i0 * G, *su = a.su + e * n + (size_t)i0 * G;
  const uint16_t* x[V];
  u32x4 tv[V][kStage];
#pragma unroll
  for (int p = 0; p < V; ++p) {
    x[p] = a.x + (size_t)(sl[p] / a.k) * a.H;
    token_load(x[p], G * 4, tid, tv[p]);
  }
  float uv[V];
  if (LORA) {
#pragma unroll
    for (int p = 0; p < V; ++p) uv[p] = a.ua[(size_t)sl[p] * 2 * a.R + min(tid, 2 * a.R - 1)];  // (R is at most 128)
  }
  u32x4 cd[kUpDepth][4];
  auto load = [&](int u, int b) {
    const uint32_t o = (u < u1 ? at + min(8 * u + c8, G - 1) : (uint32_t)i0 * G) * 16;
    cd[b][0] = buffer16<kCodes>(wg, o, 0);
    cd[b][1] = buffer16<kCodes>(wg, o, rows8);
    cd[b][2] = buffer16<kCodes>(wu, o, 0);
    cd[b][3] = buffer16<kCodes>(wu, o, rows8);
    __builtin_amdgcn_sched_barrier(0);  // (units' loads stay in order)
  };
  auto load_ahead = [&] {
#pragma unroll
    for (int b = 0; b < kUpDepth; ++b) load(u0 + b, b);
  };
  if (first_pass) {
    u32x4 sv[kStage], bv[kStage];
    stage_load<u32x4_u2>(sg, su, 2 * G, tid, sv);
    if (LORA) stage_load<u32x4>(a.bg + ((size_t)e * a.I + i0) * a.R, a.bu + ((size_t)e * a.I + i0) * a.R, 4 * a.R, tid, bv);
    __builtin_amdgcn_sched_barrier(0);
    load_ahead();
    stage_store(l.scales, 2 * G, tid, sv);
    if (LORA) stage_store(l.b, 4 * a.R, tid, bv);  // (R is at most 128: all of it)
    for (int c = 256 * kStage; c < 4 * G; c += 256 * kStage) {
      stage_load<u32x4_u2>(sg, su, 2 * G, c + tid, sv);
      stage_store(l.scales, 2 * G, c + tid, sv);
    }
  } else {
    __builtin_amdgcn_sched_barrier(0);
    load_ahead();
  }
#pragma unroll
  for (int p = 0; p < V; ++p) stage_token<MX>(l.x + p * 4 * plane, l.sums + p * Gp, G, Gp, tid, tv[p]);
  for (int c = 256 * kStage; c < 4 * Gp; c += 256 * kStage)
#pragma unroll
    for (int p = 0; p < V; ++p) {
      token_load(x[p], G * 4, c + tid, tv[p]);
      stage_token<MX>(l.x + p * 4 * plane, l.sums + p * Gp, G, Gp, c + tid, tv[p]);
    }
  if (LORA) {
#pragma unroll
    for (int p = 0; p < V; ++p)
      if (tid < 2 * a.R) l.ua[p * 2 * a.R + tid] = uv[p];
  }
  __syncthreads();
  if (LORA) {
    // B times (A x): columns by gate and up by runs of the ranks
    const int c = tid & 15, up = tid >> 4 & 1, part = tid >> 5;
    const int len = (a.R + kLoraParts - 1) / kLoraParts, r0 = part * len, n = max(min(a.R - r0, len), 0);
    float t[V] = {};
    // (a column starts its run at its own place: side by side, the columns' ranks would lie in one bank)
    int r = r0 + c % max(n, 1);
    for (int i = 0; i < n; ++i) {
#pragma unroll
      for (int p = 0; p < V; ++p) t[p] = fmaf(l.b[(up * 16 + c) * a.R + r], l.ua[(p * 2 + up) * a.R + r], t[p]);
      r = r + 1 < r0 + n ? r + 1 : r0;
    }
#pragma unroll
    for (int p = 0; p < V; ++p) l.lora[part][up][p][c] = t[p];
  }
  const DotConsts dc = dot_consts();
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
          read_vec(l.x + p * 4 * plane, g, plane, x[p]);
          sum[p] = l.sums[p * Gp + g];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float s = bf16_to_float(l.scales[(t * 8 + row) * G + min(g, G - 1)]);
          float d[V];
#pragma unroll
          for (int p = 0; p < V; ++p) d[p] = sum[p];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 w = decode8<MX>(cd[b][t][j], dc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int p = 0; p < V; ++p) d[p] = dot2<false>(w[i], x[p].v[j][i], d[p]);
          }
#pragma unroll
          for (int p = 0; p < V; ++p) acc[t][p] = fmaf(s, d[p], acc[t][p]);
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
      if (c8 == 0) l.red[t >> 1][kw][p][(t & 1) * 8 + row] = v;
    }
}

constexpr int kDownUnits = 4;           // units of a chunk of down: the loads ahead
constexpr int kDownK = kDownUnits * 8;  // its groups
constexpr int kDownPlane = kDownK * 16;
// h lies as a wave of down has it in LDS: chunks of planes of 16 bytes a group.  Bytes of a chunk, and where one is.
template <bool MX>
constexpr int kChunkBytes = (MX ? 8 : 6) * kDownPlane;
static __host__ __device__ inline size_t h_chunks(int64_t I) { return (size_t)(I / 32 + kDownK - 1) / kDownK; }
template <bool MX>
__device__ __forceinline__ size_t h_chunk(int I, int s, int chunk) {
  return ((size_t)s * h_chunks(I) + chunk) * kChunkBytes<MX>;
}
// row16_sum for integers
__device__ __forceinline__ int row16_isum(int v) {
  v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true);
  v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true);
  v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);
  return v + __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);
}

// Column i0 + c (c: the lane in its 16) of slot s from its two sums: clamp, SwiGLU, and h as down reads it.
template <bool MX, bool LORA>
__device__ __forceinline__ void finish_column(const DecodeArgs& a, float gv, float uv, int s, int i0, int c) {
  if (a.limit > 0.f) {
    // (comparisons that keep a NaN)
    gv = gv > a.limit ? a.limit : gv;
    uv = uv > a.limit ? a.limit : uv < -a.limit ? -a.limit : uv;
  }
  const float h = gv * sigmoid_f(gv) * uv;
  // brings the largest finite one of the 16 below 2^15 (118: the factor that undoes it is no subnormal)
  const bool finite = fabsf(h) < INFINITY;
  const int ex = min(pow2_exponent_for(row16_max(finite ? fabsf(h) : 0.f)), 118);
  const float hx = ldexpf(h, ex);
  const int g = i0 / 32, half = i0 >> 4 & 1;
  uint8_t* at = a.hs + h_chunk<MX>(a.I, s, g / kDownK) + (g & (kDownK - 1)) * 16;
  float2_t f;
  if (MX) {
    // fp16, and in fp16 what that left (of what is finite): planes of 8 columns
    const uint16_t hi = float_to_half_bits(hx);
    const float high = half_bits_to_float(hi);
    uint16_t* to = reinterpret_cast<uint16_t*>(at + (2 * half + (c >> 3)) * kDownPlane) + (c & 7);
    to[0] = hi;
    to[2 * kDownPlane] = float_to_half_bits(finite ? hx - high : 0.f);
    f = float2_t{0.f, ldexpf(1.f, -ex)};
  } else {
    // integers of 24 bits: planes of a byte of 16 columns, each 8 of which in the codes' order (even ones, odd ones).  One
    // that is not finite makes its 16 columns' products NaN.
    const int q = (int)rintf(fminf(fmaxf(hx * 256.f, -0x1p23f), 0x1p23f - 1.f));
    uint8_t* to = at + 3 * half * kDownPlane + ((c & 8) | (c & 1) << 2 | (c & 7) >> 1);
    to[0] = (uint8_t)q, to[kDownPlane] = (uint8_t)(q >> 8), to[2 * kDownPlane] = (uint8_t)(q >> 16);
    f = float2_t{__int_as_float(-8 * row16_isum(q)), ldexpf(1.f, -8 - ex) + row16_sum(finite ? 0.f : NAN)};
  }
  if (c == 0) a.hsf[(size_t)s * (a.I / 16) + i0 / 16] = f;
  if (LORA) a.h[(size_t)s * a.I + i0 + c] = h;
}

// bytes of dynamic LDS: V tokens, scales, and with LoRA B and ua
static __host__ __device__ inline size_t up_lds(int H, int R, int V) {
  const size_t G = (size_t)H / 32, Gp = ((G + 7) / 8 + 3) / 4 * 32;
  return V * Gp * 68 + 64 * G + (128 + 8 * V) * (size_t)R;
}

// Gate and up.  A workgroup has 16 columns of I of one expert (its first
// slot's block; the others leave at once) for all of its tokens, one or two at a time,
// which lie in LDS.  Its four waves split the contraction.  by_slot (more than two slots an expert): every
// other slot's workgroup stays, with that slot and the next.
template <bool MX, bool LORA>
__global__ __launch_bounds__(256, 4) void k_decode_gate_up(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint64_t mask[kSlotWords];
  __shared__ float red[2][4][kUpVecs][16];
  __shared__ float lora[LORA ? kLoraParts : 1][2][kUpVecs][16];
  const int slot = blockIdx.y, i0 = blockIdx.x * 16;
  const int64_t e = a.ids[slot];
  int next = -1, M = 0, rank = 0;
  Slots slots = find_slots(a, slot, e, mask, M, next, rank);
  if (a.by_slot) M = rank & 1 ? 0 : next < 0 ? 1 : 2;
  if (e < 0 || e >= a.E) M = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.next[slot] = next;
    a.lead[slot] = M > 0;
  }
  if (!M) return;
  const int G = a.H / 32, Gp = ((G + 7) / 8 + 3) / 4 * 32, V = min(kUpVecs, a.T);
  UpLds l;
  l.x = lds;
  l.sums = reinterpret_cast<float*>(lds + V * Gp * 64);
  l.scales = reinterpret_cast<uint16_t*>(l.sums + V * Gp);
  l.b = reinterpret_cast<float*>(l.scales + 32 * G);
  l.ua = l.b + 32 * a.R;
  l.red = red;
  l.lora = lora;
  // (V: a single token may name an expert twice, but LDS has room for it once)
  for (int m0 = 0; m0 < M; m0 += V) {
    const int nt = min(V, M - m0);
    int sl[kUpVecs];
    if (a.by_slot) {
      sl[0] = m0 ? next : slot, sl[1] = nt > 1 ? next : sl[0];
    } else {
      sl[0] = slots.take();
      sl[1] = nt > 1 ? slots.take() : sl[0];
    }
    if (nt == 1)
      gate_up_pass<MX, LORA, 1>(a, e, i0, sl, m0 == 0, l);
    else
      gate_up_pass<MX, LORA, kUpVecs>(a, e, i0, sl, m0 == 0, l);
    __syncthreads();
    if ((int)threadIdx.x < 16 * nt) {
      const int p = threadIdx.x >> 4, c = threadIdx.x & 15;
      const float by = MX ? 1.f : 16.f;
      float gv = by * (red[0][0][p][c] + red[0][1][p][c] + red[0][2][p][c] + red[0][3][p][c]);
      float uv = by * (red[1][0][p][c] + red[1][1][p][c] + red[1][2][p][c] + red[1][3][p][c]);
      const int s = p ? sl[1] : sl[0];
      if (LORA) {
        float lg = 0.f, lu = 0.f;
#pragma unroll
        for (int r = 0; r < kLoraParts; ++r) lg += lora[r][0][p][c], lu += lora[r][1][p][c];
        gv = fmaf(a.sc, lg, gv), uv = fmaf(a.sc, lu, uv);
      }
      finish_column<MX, LORA>(a, gv, uv, s, i0, c);
    }
    if (m0 + V < M) __syncthreads();
  }
}

// Gate and up for short rows.  There the time of the kernel above is that of its barriers and of workgroups coming and
// going, so a workgroup has 64 columns here, 16 a wave, and a wave the whole contraction: one
// barrier a pair of tokens, and what follows is each wave's own (8 tokens of 279 experts, 576 x 2016: 78 -> 58
// us; 29 of 78, 1056 x 2496: 242 -> 171; 32 of 384 on MXFP4, 2048 x 3040: 458 -> 388).  Rows are up to 2048 values (one piece
// of a token a thread, four of the scales).  Few workgroups leave units idle (one token, 2048 x 1024: 22.2 us, here
// 22.8; two, 2048 x 512: 16.3 and 16.8; one, 1024 x 2048: 16.8 and 14.8), and rows of B above rank 64 are better
// shared through LDS (16 tokens, rank 128, 1024 x 512: 108, here 117).
constexpr int kShort = 2048, kShortRank = 64;
constexpr int64_t kShortColumns = 12288;  // of all slots

template <bool MX, bool LORA, int V>
__device__ __forceinline__ void gate_up_short(const DecodeArgs& a, int64_t e, int i0, int columns, const int* sl, bool rows,
                                              const UpLds& l) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c8 = lane & 7, row = lane >> 3;
  const int G = a.H / 32, units = (G + 7) / 8, Gp = units * 8, plane = Gp * 16;
  const size_t n = (size_t)a.I * G;
  const Buffer wg = buffer_of(a.wg + e * n * 16, n * 16), wu = buffer_of(a.wu + e * n * 16, n * 16);
  // (a wave behind the last column reads the last 16)
  const int j0 = min(i0 + 16 * kw, a.I - 16);
  const uint32_t at = (uint32_t)(j0 + row) * G, rows8 = 128u * G;
  u32x4 tv[V], sv[kStage];
  float uv[V];
#pragma unroll
  for (int p = 0; p < V; ++p)  // (a row has at most 256 pieces)
    tv[p] = *(reinterpret_cast<const u32x4*>(a.x + (size_t)(sl[p] / a.k) * a.H) + min(tid, G * 4 - 1));
  if (LORA) {
#pragma unroll
    for (int p = 0; p < V; ++p) uv[p] = a.ua[(size_t)sl[p] * 2 * a.R + min(tid, 2 * a.R - 1)];
  }
  const int pieces = columns * G / 8;
  if (rows) stage_load<u32x4_u2>(a.sg + e * n + (size_t)i0 * G, a.su + e * n + (size_t)i0 * G, pieces, tid, sv);
  __builtin_amdgcn_sched_barrier(0);
  u32x4 cd[kUpDepth][4];
  auto load = [&](int u, int b) {
    const uint32_t o = (u < units ? at + min(8 * u + c8, G - 1) : (uint32_t)j0 * G) * 16;
    cd[b][0] = buffer16<kCodes>(wg, o, 0);
    cd[b][1] = buffer16<kCodes>(wg, o, rows8);
    cd[b][2] = buffer16<kCodes>(wu, o, 0);
    cd[b][3] = buffer16<kCodes>(wu, o, rows8);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int b = 0; b < kUpDepth; ++b) load(b, b);
  if (rows) stage_store(l.scales, pieces, tid, sv);
#pragma unroll
  for (int p = 0; p < V; ++p) {
    u32x4 w = tv[p];
    if (tid >= G * 4) w = u32x4{0, 0, 0, 0};
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) s += bf_lo(w[j]) + bf_hi(w[j]);
    s += dpp_f<0xB1>(s);
    s += dpp_f<0x4E>(s);
    if (tid < Gp * 4) {
      *reinterpret_cast<u32x4*>(l.x + p * 4 * plane + ((tid & 3) * Gp + (tid >> 2)) * 16) = MX ? w : order8(w);
      if ((tid & 3) == 0) l.sums[p * Gp + (tid >> 2)] = MX ? 0.f : -1.5f * s;
    }
    if (LORA && tid < 2 * a.R) l.ua[p * 2 * a.R + tid] = uv[p];
  }
  __syncthreads();
  float lg[V] = {}, lu[V] = {};
  if (LORA) {
    // B times (A x): a lane takes every fourth rank of a column
    const int c = lane & 15;
    const float *bg = a.bg + ((size_t)e * a.I + j0 + c) * a.R, *bu = a.bu + ((size_t)e * a.I + j0 + c) * a.R;
#pragma unroll 4
    for (int r = lane >> 4; r < a.R; r += 4) {
      const float g = bg[r], u = bu[r];
#pragma unroll
      for (int p = 0; p < V; ++p) {
        lg[p] = fmaf(g, l.ua[p * 2 * a.R + r], lg[p]);
        lu[p] = fmaf(u, l.ua[(p * 2 + 1) * a.R + r], lu[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < V; ++p) lg[p] = rows_sum(lg[p]), lu[p] = rows_sum(lu[p]);
  }
  const DotConsts dc = dot_consts();
  const uint16_t* sc = l.scales + (j0 - i0 + row) * G;
  float acc[4][V] = {};
  for (int v = 0; v < units; v += kUpDepth) {
#pragma unroll
    for (int b = 0; b < kUpDepth; ++b) {
      if (v + b < units) {
        const int g = 8 * (v + b) + c8;
        Vec x[V];
        float sum[V];
#pragma unroll
        for (int p = 0; p < V; ++p) {
          read_vec(l.x + p * 4 * plane, g, plane, x[p]);
          sum[p] = l.sums[p * Gp + g];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float s = bf16_to_float(sc[((t >> 1) * columns + (t & 1) * 8) * G + min(g, G - 1)]);
          float d[V];
#pragma unroll
          for (int p = 0; p < V; ++p) d[p] = sum[p];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 w = decode8<MX>(cd[b][t][j], dc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int p = 0; p < V; ++p) d[p] = dot2<false>(w[i], x[p].v[j][i], d[p]);
          }
#pragma unroll
          for (int p = 0; p < V; ++p) acc[t][p] = fmaf(s, d[p], acc[t][p]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      load(v + b + kUpDepth, b);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int p = 0; p < V; ++p) {
      const float v = eight_sum(acc[t][p]);
      if (c8 == 0) l.red[t >> 1][kw][p][(t & 1) * 8 + row] = v;
    }
  wave_fence();
  if (lane < 16 * V && 16 * kw < columns) {
    const int c = lane & 15, p = lane >> 4;
    const float by = MX ? 1.f : 16.f;
    float gv = by * l.red[0][kw][p][c], uw = by * l.red[1][kw][p][c];
    if (LORA) gv = fmaf(a.sc, V > 1 && p ? lg[V - 1] : lg[0], gv), uw = fmaf(a.sc, V > 1 && p ? lu[V - 1] : lu[0], uw);
    finish_column<MX, LORA>(a, gv, uw, p ? sl[V - 1] : sl[0], j0, c);
  }
}

// bytes of dynamic LDS: V tokens, scales of 64 columns, and with LoRA ua
static __host__ __device__ inline size_t short_lds(int H, int R, int V) {
  const size_t G = (size_t)H / 32, Gp = (G + 7) / 8 * 8;
  return V * Gp * 68 + 256 * G + 8 * (size_t)V * R;
}

template <bool MX, bool LORA>
__global__ __launch_bounds__(256, 4) void k_decode_gate_up_short(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint64_t mask[kSlotWords];
  __shared__ float red[2][4][kUpVecs][16];
  const int slot = blockIdx.y, i0 = blockIdx.x * 64, columns = min(64, a.I - i0);
  const int64_t e = a.ids[slot];
  int next = -1, M = 0, rank = 0;
  Slots slots = find_slots(a, slot, e, mask, M, next, rank);
  if (a.by_slot) M = rank & 1 ? 0 : next < 0 ? 1 : 2;
  if (e < 0 || e >= a.E) M = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.next[slot] = next;
    a.lead[slot] = M > 0;
  }
  if (!M) return;
  const int G = a.H / 32, Gp = (G + 7) / 8 * 8, V = min(kUpVecs, a.T);
  UpLds l{};
  l.x = lds;
  l.sums = reinterpret_cast<float*>(lds + V * Gp * 64);
  l.scales = reinterpret_cast<uint16_t*>(l.sums + V * Gp);
  l.ua = reinterpret_cast<float*>(l.scales + 128 * G);
  l.red = red;
  // (V: a single token may name an expert twice, but LDS has room for it once)
  for (int m0 = 0; m0 < M; m0 += V) {
    const int nt = min(V, M - m0);
    int sl[kUpVecs];
    if (a.by_slot) {
      sl[0] = m0 ? next : slot, sl[1] = nt > 1 ? next : sl[0];
    } else {
      sl[0] = slots.take();
      sl[1] = nt > 1 ? slots.take() : sl[0];
    }
    if (nt == 1)
      gate_up_short<MX, LORA, 1>(a, e, i0, columns, sl, m0 == 0, l);
    else
      gate_up_short<MX, LORA, kUpVecs>(a, e, i0, columns, sl, m0 == 0, l);
    if (m0 + V < M) __syncthreads();
  }
}

// A row of A times V tokens' vectors (bf16 x, or fp32 h), by a wave: 1024 values in flight a vector.
template <bool DOWN, int V>
__device__ __forceinline__ void lora_row(const DecodeArgs& a, const float* w, const int* sl, float* out, int pitch) {
  const int K = DOWN ? a.I : a.H, lane = threadIdx.x & 63;
  float v[V] = {};
  for (int c0 = lane * 4; c0 < K; c0 += 1024) {
    float4 b[4], x[4][V];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (values behind the row's end: its last ones, times 0)
      const int c = min(c0 + 256 * i, K - 4);
      b[i] = *reinterpret_cast<const float4*>(w + c);
#pragma unroll
      for (int p = 0; p < V; ++p) {
        if (DOWN) {
          x[i][p] = *reinterpret_cast<const float4*>(a.h + (size_t)sl[p] * K + c);
        } else {
          const u32pair t = *reinterpret_cast<const u32pair*>(a.x + (size_t)(sl[p] / a.k) * K + c);
          x[i][p] = float4{bf_lo(t.x), bf_hi(t.x), bf_lo(t.y), bf_hi(t.y)};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c0 + 256 * i >= K) b[i] = float4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < V; ++p) {
        v[p] = fmaf(b[i].x, x[i][p].x, v[p]);
        v[p] = fmaf(b[i].y, x[i][p].y, v[p]);
        v[p] = fmaf(b[i].z, x[i][p].z, v[p]);
        v[p] = fmaf(b[i].w, x[i][p].w, v[p]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < V; ++p) {
    const float t = wave_sum(v[p]);
    if (lane == 0) out[(size_t)sl[p] * pitch] = t;
  }
}

// x A_g^T | x A_u^T of every slot (DOWN: h A_d^T): a wave per row of A of an expert, for all of its tokens, one or two at a time.
template <bool DOWN>
__global__ __launch_bounds__(256) void k_decode_lora_a(DecodeArgs a) {
  __shared__ uint64_t mask[kSlotWords];
  const int64_t e = a.ids[blockIdx.y];
  int next, M, rank;
  Slots slots = find_slots(a, blockIdx.y, e, mask, M, next, rank);
  if (!M || e < 0 || e >= a.E) return;
  const int rows = DOWN ? a.R : 2 * a.R, r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int K = DOWN ? a.I : a.H;
  const float* w = (DOWN ? a.ad : r < a.R ? a.ag : a.au) + ((size_t)e * a.R + (r < a.R ? r : r - a.R)) * K;
  float* out = (DOWN ? a.ud : a.ua) + r;
  for (int m = 0; m < M; m += 2) {
    int sl[2];
    sl[0] = slots.take();
    if (m + 1 < M) {
      sl[1] = slots.take();
      lora_row<DOWN, 2>(a, w, sl, out, rows);
    } else {
      lora_row<DOWN, 1>(a, w, sl, out, rows);
    }
  }
}

// 16 codes times their h (x: its planes, of MXFP4 the second fp16 numbers four planes on).
template <bool MX>
__device__ __forceinline__ float half_product(uint32_t w0, uint32_t w1, const u32x4* x, uint32_t sum) {
  const uint32_t w[2] = {w0, w1};
  if (MX) {
    float d = 0.f, l = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 v = decode8_mx<true>(w[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) d = dot2<true>(v[j], x[i][j], d), l = dot2<true>(v[j], x[4 + i][j], l);
    }
    return d + l;
  }
  // (32 bits hold the whole: 15 x 16 x 2^23; the parts may wrap)
  uint32_t d0 = sum, d1 = 0;
  int d2 = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t c[2] = {w[i] & 0x0f0f0f0fu, w[i] >> 4 & 0x0f0f0f0fu};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      d0 = __builtin_amdgcn_udot4(c[j], x[0][2 * i + j], d0, false);
      d1 = __builtin_amdgcn_udot4(c[j], x[1][2 * i + j], d1, false);
      d2 = __builtin_amdgcn_sdot4((int)c[j], (int)x[2][2 * i + j], d2, false);
    }
  }
  return (float)(int)(((((uint32_t)d2 << 8) + d1) << 8) + d0);
}

constexpr int kDownWaves = 8;
template <bool MX>
constexpr int kDownLds = kChunkBytes<MX> + kDownK * (16 + 32);  // bytes a wave: h, sums and factors, scales of 16 rows

// bytes of dynamic LDS (64 tokens of 8 slots each leave room for a second workgroup)
template <bool MX>
static inline size_t down_lds(int T, int S) {
  return kDownWaves * (kDownLds<MX> + (size_t)T * 64) + (size_t)(S + 63) / 64 * 64 * 6;
}

// Down and the sum over the slots.  A workgroup has 16 columns of H; its waves
// take the experts in turn (a wave per expert, the whole contraction), a slot at a
// time, and add to sums of their own per token, which the end joins in the waves'
// order.  Where that leaves the chip idle, the experts are split over the grid's y too,
// with sums that k_decode_join adds, and by_slot a wave takes single slots.  A wave goes through its slots' contractions in chunks without a stop:
// while it multiplies one, the codes, scales and h of the next are on their way.
template <bool MX, bool LORA>
__global__ __launch_bounds__(64 * kDownWaves, 4) void k_decode_down(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c8 = lane & 7, row = lane >> 3;
  const int h0 = blockIdx.x * 16, G = a.I / 32;
  constexpr int kLoads = kChunkBytes<MX> / 1024;  // of h, a chunk
  uint8_t* hl = lds + wave * kDownLds<MX>;                         // planes of h
  u32x4* sf = reinterpret_cast<u32x4*>(hl + kChunkBytes<MX>);      // [group]: sum and factor of its halves
  uint16_t* sl = reinterpret_cast<uint16_t*>(sf + kDownK);         // [16][kDownK] scales
  float* acc = reinterpret_cast<float*>(lds + kDownWaves * kDownLds<MX>);  // [waves][T][16]
  // the experts' first slots, in order
  __shared__ uint64_t mask[kSlotWords];
  const int words = (a.S + 63) / 64;
  uint16_t* order = reinterpret_cast<uint16_t*>(acc + kDownWaves * a.T * 16);  // [words][64], as the next two
  uint16_t* expert = order + words * 64;
  int16_t* next = reinterpret_cast<int16_t*>(expert + words * 64);
  for (int w = wave; w < words; w += kDownWaves) {
    const int s = w * 64 + lane, i = min(s, a.S - 1);
    const int lead = a.lead[i], after = a.next[i], id = (int)a.ids[i];
    const uint64_t m = __ballot(s < a.S && (a.by_slot ? a.ids[i] >= 0 && a.ids[i] < a.E : lead));
    if (lane == 0) mask[w] = m;
    next[s] = (int16_t)(a.by_slot ? -1 : after);
    expert[s] = (uint16_t)id;
  }
  for (int i = threadIdx.x; i < kDownWaves * a.T * 16; i += 64 * kDownWaves) acc[i] = 0.f;
  __syncthreads();
  int U = 0;
  for (int w = 0; w < words; ++w) {
    const uint64_t m = mask[w];
    if ((w & (kDownWaves - 1)) == wave && (m >> lane & 1)) order[U + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(w * 64 + lane);
    U += __popcll(m);
  }
  __syncthreads();
  const int first = blockIdx.y * kDownWaves + wave, stride = gridDim.y * kDownWaves;
  if (first < U) {
    const Buffer hb = buffer_of(a.hs, h_chunk<MX>(a.I, a.S, 0)), fb = buffer_of(a.hsf, (size_t)a.S * (a.I / 16) * 8);
    const uint32_t at = (uint32_t)(h0 + row) * G, rows8 = 128u * G;
    const size_t n = (size_t)a.H * G;
    // the chunk whose loads are issued next
    int j = first, s = __builtin_amdgcn_readfirstlane(order[j]), k0 = 0;
    size_t e = __builtin_amdgcn_readfirstlane(expert[s]);
    bool more = true;  // (there is one)
    u32x4 cd[kDownUnits][2], hn[kLoads], sn;
    float2_t fn;
    auto load_codes = [&](int b) {
      const Buffer w = buffer_of(a.wd + e * n * 16, n * 16);
      const uint32_t o = (more ? at + min(k0 + 8 * b + c8, G - 1) : (uint32_t)h0 * G) * 16;
      cd[b][0] = buffer16<kCodes>(w, o, 0);
      cd[b][1] = buffer16<kCodes>(w, o, rows8);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto load_rest = [&] {
      // scales: a lane has 8 groups of one of the 16 rows
      const int l = more ? lane : 0;
      const uint16_t* p = a.sd + e * n + (size_t)(h0 + (l >> 2)) * G;
      const int g = k0 + (l & 3) * 8;
      if (k0 + kDownK <= G) {
        sn = *reinterpret_cast<const u32x4_u2*>(p + g);
      } else {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[min(g + i, G - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) sn[i] = v[2 * i] | v[2 * i + 1] << 16;
      }
      // h as it lies; sums and factors: halves of groups
      const uint32_t ho = (uint32_t)h_chunk<MX>(a.I, s, k0 / kDownK) + l * 16;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) hn[i] = buffer16<kKept>(hb, ho + 1024 * i, 0);
      const uint32_t fo = min(((uint32_t)s * G + k0) * 16 + l * 8, (uint32_t)(s + 1) * G * 16 - 8);
      fn = __builtin_bit_cast(float2_t, __builtin_amdgcn_raw_buffer_load_b64(fb, (int)fo, 0, 0));
      __builtin_amdgcn_sched_barrier(0);
    };
    load_rest();
#pragma unroll
    for (int b = 0; b < kDownUnits; ++b) load_codes(b);
    float y[2] = {0.f, 0.f};
    while (more) {
      // this chunk's h, sums, factors and scales to LDS, 0 behind the contraction's end
      const int cs = s, ck = k0, len = min(kDownK, G - ck);
      const size_t ce = e;
      const u32x4 zero = {0, 0, 0, 0};
      wave_fence();
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        *reinterpret_cast<u32x4*>(hl + (lane + 64 * i) * 16) = (lane & (kDownK - 1)) < len ? hn[i] : zero;
      reinterpret_cast<float2_t*>(sf)[lane] = lane < 2 * len ? fn : float2_t{0.f, 0.f};
      *reinterpret_cast<u32x4*>(sl + lane * 8) = sn;
      wave_fence();
      // the next one
      k0 += kDownK;
      if (k0 >= G) {
        k0 = 0;
        int t = __builtin_amdgcn_readfirstlane(next[s]);
        if (t < 0) {
          j += stride;
          more = j < U;
          if (more) {
            t = __builtin_amdgcn_readfirstlane(order[j]);
            e = __builtin_amdgcn_readfirstlane(expert[t]);
          } else {
            t = s;
          }
        }
        s = t;
      }
      load_rest();
      const int units = (len + 7) / 8;
#pragma unroll
      for (int b = 0; b < kDownUnits; ++b) {
        if (b < units) {
          const int g = 8 * b + c8;
          const u32x4 f = sf[g];
          u32x4 x[kChunkBytes<MX> / kDownPlane];
#pragma unroll
          for (int j = 0; j < kChunkBytes<MX> / kDownPlane; ++j)
            x[j] = *reinterpret_cast<const u32x4*>(hl + j * kDownPlane + g * 16);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float d[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) d[h] = half_product<MX>(cd[b][t][2 * h], cd[b][t][2 * h + 1], x + (MX ? 2 : 3) * h, f[2 * h]);
            const float sc = bf16_to_float(sl[(t * 8 + row) * kDownK + g]);
            y[t] = fmaf(sc, fmaf(__uint_as_float(f.y), d[0], __uint_as_float(f.w) * d[1]), y[t]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        load_codes(b);
      }
      if (ck + kDownK < G) continue;
      // the slot is done
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float v = eight_sum(y[t]);
        y[t] = 0.f;
        if (LORA) {
          // an eighth of the ranks a lane
          const float *b = a.bd + (ce * a.H + h0 + 8 * t + row) * a.R, *u = a.ud + (size_t)cs * a.R;
          float l = 0.f;
#pragma unroll 2
          for (int r = c8; r < a.R; r += 8) l = fmaf(b[r], u[r], l);
          v = fmaf(a.sc, eight_sum(l), v);
        }
        if (c8 == 0) {
          float* o = acc + (wave * a.T + cs / a.k) * 16 + 8 * t + row;
          *o = fmaf(a.rw[cs], v, *o);
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += 64 * kDownWaves) {
    float v = 0.f;
    for (int w = 0; w < kDownWaves; ++w) v += acc[w * a.T * 16 + i];
    const size_t o = (size_t)(i >> 4) * a.H + h0 + (i & 15);
    if (gridDim.y == 1)
      a.out[o] = float_to_bf16(v);
    else
      a.part[(size_t)blockIdx.y * a.T * a.H + o] = v;
  }
}

__global__ __launch_bounds__(256) void k_decode_join(DecodeArgs a, int parts) {
  const int n = a.T * a.H, i = (blockIdx.x * 256 + threadIdx.x) * 4;  // (H is a multiple of 32)
  if (i >= n) return;
  floatx4 v = *reinterpret_cast<const floatx4*>(a.part + i);
#pragma unroll 4
  for (int p = 1; p < parts; ++p) v += *reinterpret_cast<const floatx4*>(a.part + (size_t)p * n + i);
  *reinterpret_cast<u32pair_u2*>(a.out + i) = u32pair{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
}

// ---------------------------------------------------------------- host

static bool down_by_slot(int64_t E, int64_t S) { return S > 2 * E; }

// Down's parts: two workgroups a unit of the chip, as far as experts or slots reach (8 tokens of 279 experts, 576 x 2016: 116 -> 79 us;
// 11 of 272, 416 x 1280, rank 64: 182 -> 100).  256 blocks of columns, a workgroup a unit, are not split: 4 tokens with rank 16 at
// hidden 4096 96 us both ways, 4128 131 (split 127), 6144 144 both ways, 7168 154 (158); 8 slots or fewer are one workgroup's in any case.
static int down_parts(int64_t H, int64_t E, int64_t S) {
  const int64_t units = down_by_slot(E, S) || S < E ? S : E, columns = H / 16;  // (experts or slots for the waves, at most)
  const int64_t want = (512 + columns - 1) / columns, most = (units + kDownWaves - 1) / kDownWaves;
  return (int)(columns >= 256 ? 1 : want < most ? want : most);
}

struct DecodePlan {
  size_t hs, hsf, h, next, lead, ua, ud, part, total;
};
static DecodePlan plan_decode(const Dims& d) {
  DecodePlan p;
  const size_t S = (size_t)d.Ms;
  p.next = 0;
  p.lead = round256(4 * S);
  p.hs = p.lead + round256(4 * S);
  p.hsf = p.hs + round256(S * h_chunks(d.I) * (d.fmt == KT_RAWINT4_FORMAT_MXFP4 ? kChunkBytes<true> : kChunkBytes<false>));
  p.h = p.hsf + round256(8 * S * (d.I / 16));
  p.ua = p.h + (d.R ? round256(4 * S * d.I) : 0);
  p.ud = p.ua + round256(4 * S * 2 * d.R);
  p.part = p.ud + round256(4 * S * d.R);
  const int parts = S ? down_parts(d.H, d.E, d.Ms) : 1;
  p.total = p.part + (parts > 1 ? round256((size_t)4 * parts * d.qlen * d.H) : 0);
  return p;
}

static int check_decode(const kt_rawint4_moe_layer* layer, int32_t tokens, Dims* d) {
  const int rc = check_layer_dims(layer, tokens, d, true);
  if (rc) return rc;
  if (layer->hidden > KT_MOE_DECODE_MAX_HIDDEN) return set_error(KT_RAWINT4_EINVAL, "hidden must be at most 16384");
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
  const int V = a.T < kUpVecs ? a.T : kUpVecs;
  if (a.H <= kShort && a.R <= kShortRank && (int64_t)a.I * a.S >= kShortColumns)
    k_decode_gate_up_short<MX, LORA><<<dim3((unsigned)((a.I + 63) / 64), (unsigned)a.S), 256, short_lds(a.H, a.R, V), st>>>(a);
  else
    k_decode_gate_up<MX, LORA><<<dim3((unsigned)(a.I / 16), (unsigned)a.S), 256, up_lds(a.H, a.R, V), st>>>(a);
  note_launch();
  if (LORA) {
    k_decode_lora_a<true><<<dim3((unsigned)((a.R + 3) / 4), (unsigned)a.S), 256, 0, st>>>(a);
    note_launch();
  }
  const int parts = down_parts(a.H, a.E, a.S);
  k_decode_down<MX, LORA>
      <<<dim3((unsigned)(a.H / 16), (unsigned)parts), 64 * kDownWaves, down_lds<MX>(a.T, a.S), st>>>(a);
  note_launch();
  if (parts > 1) {
    k_decode_join<<<(unsigned)((a.T * a.H / 4 + 255) / 256), 256, 0, st>>>(a, parts);
    note_launch();
  }
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
  a.hs = ws_ptr<uint8_t>(workspace, p.hs);
  a.hsf = ws_ptr<float2_t>(workspace, p.hsf);
  a.next = ws_ptr<int32_t>(workspace, p.next);
  a.lead = ws_ptr<int32_t>(workspace, p.lead);
  a.ua = ws_ptr<float>(workspace, p.ua);
  a.ud = ws_ptr<float>(workspace, p.ud);
  a.part = ws_ptr<float>(workspace, p.part);
  // (more than two slots an expert on average: codes come from the caches all the same, and one workgroup after the other would
  // wait for the longest list; 21 tokens of 4 experts, 160 x 1216: 85 -> 65 us, 13 of 8, 6880 x 2912: 205 -> 193)
  a.by_slot = down_by_slot(a.E, a.S);
  hipStream_t st = static_cast<hipStream_t>(stream);
  begin_launches();
  if (d.fmt == KT_RAWINT4_FORMAT_MXFP4)
    d.R ? launch_decode<true, true>(a, st) : launch_decode<true, false>(a, st);
  else
    d.R ? launch_decode<false, true>(a, st) : launch_decode<false, false>(a, st);
  return finish_launches();
}

}  // extern "C"
