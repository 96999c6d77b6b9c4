// Activation checkpoints in 8 bits: bf16 rows as one byte per value and one
// power-of-two exponent byte per 32 columns of a row, and back.
//
// With amax the group's largest magnitude, the exponent e is the smallest at
// which no code overflows:
//   INT8   rne(amax * 2^-e) <= 127:  amax = m * 2^x (1 <= m < 2) gives e = x - 6,
//          or x - 5 where m * 64 rounds to 128 (m = 1 + 127/128, the largest bf16
//          significand);
//   E4M3   amax * 2^-e <= 448 = 1.75 * 2^8:  e = x - 8, or x - 7 where m > 1.75.
// Multiplying by 2^-e is exact in fp32, so the only rounding is the one to the
// code.  Where that would round a value beyond bf16's largest number, the next
// code below is taken: groups with x = 127 keep INT8's exponent at 121 with
// codes up to 127, and E4M3's exponent of 120 holds codes to 240.  A code has at most 7 (INT8) or 4 (E4M3) significant bits, fewer than
// bf16's 8, so unpacking rounds nothing.
#include "kt_common.hpp"
#include "kt_internal.hpp"

namespace kt {

// 2^e for -127 <= e <= 127 (e = -127 is the subnormal 2^-127)
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(e > -127 ? (uint32_t)(e + 127) << 23 : 1u << 22); }

// Scale byte of a group from its largest magnitude's fp32 bits (a bf16 value,
// sign cleared): 255 for infinities and NaNs.
template <int FMT>
__device__ __forceinline__ int ckpt8_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255;
  if (amax == 0) return 0;
  int x = (int)(amax >> 23);  // biased exponent
  uint32_t frac = amax & 0x7fffffu;
  if (x == 0) return 0;  // subnormal: every exponent below -127 is -127
  const int e = FMT == KT_CKPT8_INT8 ? x - 6 + (frac >= 0x7f0000u && x < 254) : x - 8 + (frac > 0x600000u);
  return e > 0 ? e : 0;
}

// The largest code magnitude of a group with scale byte s.
template <int FMT>
__device__ __forceinline__ float ckpt8_limit(int s) {
  return FMT == KT_CKPT8_INT8 ? 127.f : s == 247 ? 240.f : 448.f;
}

// One value: code byte of v * inv (inv = 2^-e).
template <int FMT>
__device__ __forceinline__ uint32_t ckpt8_code(float v, float inv, float limit) {
  const float c = fminf(fmaxf(v * inv, -limit), limit);
  if (FMT == KT_CKPT8_INT8) return (uint32_t)(int)rintf(c) & 0xffu;
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, 0.f, 0, false) & 0xffu;
}

// The scale a byte stands for; NaN for 255.
__device__ __forceinline__ float ckpt8_mult(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : pow2f(byte - 127);
}

// Two neighbouring lanes share a group, 16 values each: two 16-byte loads and
// one 16-byte store a lane.  FLAT: rows are whole groups, so the tensor is one
// run of groups.  Otherwise rows start at any 2-byte (codes: 1-byte) address, for
// which the hardware's unaligned accesses serve as well, and the last group
// of a row, if it is shorter, goes value by value.  Bound by memory: 16384 x 7168
// packs in 80 us (4.4 TB/s) and unpacks in 71 us (5.0), where a plain copy of 1
// GiB reaches 5.1; half a wave a group, one value a lane, took 457 us for both.
struct Ckpt8Args {
  int64_t rows, cols, ng;  // ng: groups per row
  const uint16_t* x;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* y;
};

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x4 u32x4_byte __attribute__((aligned(1)));

// start of half group i (2 per group) in the tensor and how many of its 16 values exist
template <bool FLAT>
__device__ __forceinline__ int64_t half_group(const Ckpt8Args& a, int64_t i, int& n) {
  if (FLAT) {
    n = 16;
    return i * 16;
  }
  const int64_t g = i >> 1;
  int64_t row;
  if (a.rows * a.ng < ((int64_t)1 << 31))
    row = (uint32_t)g / (uint32_t)a.ng;
  else
    row = g / a.ng;
  const int64_t c = (g - row * a.ng) * 32 + (i & 1) * 16, left = a.cols - c;
  n = left >= 16 ? 16 : left > 0 ? (int)left : 0;
  return row * a.cols + c;
}

template <int FMT, bool FLAT, int UNITS>
__global__ __launch_bounds__(256) void k_ckpt8_pack(Ckpt8Args a) {
  const int64_t total = a.rows * a.ng * 2, i0 = (int64_t)blockIdx.x * (256 * UNITS) + threadIdx.x;
  uint32_t w[UNITS][8];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int64_t i = i0 + u * 256;
#pragma unroll
    for (int q = 0; q < 8; ++q) w[u][q] = 0;
    if (i >= total) continue;
    int n;
    const int64_t at = half_group<FLAT>(a, i, n);
    if (FLAT || n == 16) {
      const u32x4 p = *reinterpret_cast<const u32x4_any*>(a.x + at), q = *reinterpret_cast<const u32x4_any*>(a.x + at + 8);
      w[u][0] = p.x, w[u][1] = p.y, w[u][2] = p.z, w[u][3] = p.w;
      w[u][4] = q.x, w[u][5] = q.y, w[u][6] = q.z, w[u][7] = q.w;
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (q < n) w[u][q >> 1] |= (uint32_t)a.x[at + q] << (16 * (q & 1));
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int64_t i = i0 + u * 256;
    uint32_t hi = 0, lo = 0;  // largest magnitudes of the high and low halves
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      hi = max(hi, w[u][q] & 0x7fff0000u);
      lo = max(lo, w[u][q] & 0x7fffu);
    }
    uint32_t amax = max(hi, lo << 16);
    // the other lane of the group (both are in the range or neither)
    amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0xB1, 0xf, 0xf, true));
    if (i >= total) continue;
    const int s = ckpt8_scale<FMT>(amax);
    const float inv = s == 255 ? 0.f : pow2f(127 - s), limit = ckpt8_limit<FMT>(s);
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t v = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t d = w[u][2 * q + h];
        v |= (ckpt8_code<FMT>(__uint_as_float(d << 16), inv, limit) |
              ckpt8_code<FMT>(__uint_as_float(d & 0xffff0000u), inv, limit) << 8)
             << (16 * h);
      }
      c[q] = s == 255 ? 0u : v;
    }
    int n;
    const int64_t at = half_group<FLAT>(a, i, n);
    if (FLAT || n == 16) {
      *reinterpret_cast<u32x4_byte*>(a.codes + at) = u32x4{c[0], c[1], c[2], c[3]};
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (q < n) a.codes[at + q] = (uint8_t)(c[q >> 2] >> (8 * (q & 3)));
    }
    if ((i & 1) == 0) a.scales[i >> 1] = (uint8_t)s;
  }
}

// Two values of a code dword (low or high half) times the group's scale as two bf16.
template <int FMT, bool HIGH>
__device__ __forceinline__ uint32_t ckpt8_pair(uint32_t c, float mult) {
  float v0, v1;
  if (FMT == KT_CKPT8_INT8) {
    v0 = (float)(int8_t)(c >> (HIGH ? 16 : 0));
    v1 = (float)(int8_t)(c >> (HIGH ? 24 : 8));
  } else {
    const float2_t f = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, HIGH);
    v0 = f.x;
    v1 = f.y;
  }
  v0 *= mult;
  v1 *= mult;
  return pack2(float_to_bf16(v0), float_to_bf16(v1));
}

template <int FMT, bool FLAT, int UNITS>
__global__ __launch_bounds__(256) void k_ckpt8_unpack(Ckpt8Args a) {
  const int64_t total = a.rows * a.ng * 2, i0 = (int64_t)blockIdx.x * (256 * UNITS) + threadIdx.x;
  uint32_t c[UNITS][4];
  int s[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int64_t i = i0 + u * 256;
#pragma unroll
    for (int q = 0; q < 4; ++q) c[u][q] = 0;
    s[u] = 0;
    if (i >= total) continue;
    s[u] = a.scales[i >> 1];
    int n;
    const int64_t at = half_group<FLAT>(a, i, n);
    if (FLAT || n == 16) {
      const u32x4 v = *reinterpret_cast<const u32x4_byte*>(a.codes + at);
      c[u][0] = v.x, c[u][1] = v.y, c[u][2] = v.z, c[u][3] = v.w;
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (q < n) c[u][q >> 2] |= (uint32_t)a.codes[at + q] << (8 * (q & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int64_t i = i0 + u * 256;
    if (i >= total) continue;
    const float mult = ckpt8_mult(s[u]);
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      o[2 * q] = ckpt8_pair<FMT, false>(c[u][q], mult);
      o[2 * q + 1] = ckpt8_pair<FMT, true>(c[u][q], mult);
    }
    int n;
    const int64_t at = half_group<FLAT>(a, i, n);
    if (FLAT || n == 16) {
      *reinterpret_cast<u32x4_any*>(a.y + at) = u32x4{o[0], o[1], o[2], o[3]};
      *reinterpret_cast<u32x4_any*>(a.y + at + 8) = u32x4{o[4], o[5], o[6], o[7]};
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (q < n) a.y[at + q] = (uint16_t)(o[q >> 1] >> (16 * (q & 1)));
    }
  }
}

template <int FMT, bool FLAT, int UNITS>
static void launch_ckpt8_as(const Ckpt8Args& a, bool pack, hipStream_t st) {
  const int64_t blocks = (a.rows * a.ng * 2 + 256 * UNITS - 1) / (256 * UNITS);
  if (pack)
    k_ckpt8_pack<FMT, FLAT, UNITS><<<(unsigned)blocks, 256, 0, st>>>(a);
  else
    k_ckpt8_unpack<FMT, FLAT, UNITS><<<(unsigned)blocks, 256, 0, st>>>(a);
  note_launch();
}

template <int FMT, bool FLAT>
static void launch_ckpt8_units(const Ckpt8Args& a, bool pack, hipStream_t st) {
  // four units a thread keep more loads in flight once the chip is full without them (2^21 half groups: 8 waves a SIMD)
  if (a.rows * a.ng * 2 >= (int64_t)8 * 256 * 1024)
    launch_ckpt8_as<FMT, FLAT, 4>(a, pack, st);
  else
    launch_ckpt8_as<FMT, FLAT, 1>(a, pack, st);
}

static void launch_ckpt8(Ckpt8Args a, int format, bool pack, hipStream_t st) {
  a.ng = (a.cols + 31) / 32;
  if (a.rows * a.ng == 0) return;
  const bool flat = a.cols % 32 == 0;
  if (format == KT_CKPT8_INT8) {
    if (flat)
      launch_ckpt8_units<KT_CKPT8_INT8, true>(a, pack, st);
    else
      launch_ckpt8_units<KT_CKPT8_INT8, false>(a, pack, st);
  } else {
    if (flat)
      launch_ckpt8_units<KT_CKPT8_E4M3, true>(a, pack, st);
    else
      launch_ckpt8_units<KT_CKPT8_E4M3, false>(a, pack, st);
  }
}

static void launch_ckpt8_pack(const uint16_t* x, int64_t rows, int64_t cols, int format, uint8_t* codes,
                              uint8_t* scales, hipStream_t st) {
  launch_ckpt8({rows, cols, 0, x, codes, scales, nullptr}, format, true, st);
}

void launch_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int format,
                         uint16_t* x, hipStream_t st) {
  launch_ckpt8({rows, cols, 0, nullptr, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), x}, format, false,
               st);
}

static int check_ckpt8(const void* x, int64_t rows, int64_t cols, int32_t format, const void* codes,
                       const void* scales) {
  if (rows < 0 || cols < 0 || cols > ((int64_t)1 << 32) || (cols > 0 && rows > ((int64_t)1 << 32) / ((cols + 31) / 32)))
    return set_error(KT_RAWINT4_EINVAL, "rows and cols must be non-negative, the groups at most 2^32");
  if (format != KT_CKPT8_INT8 && format != KT_CKPT8_E4M3)
    return set_error(KT_RAWINT4_EINVAL, "format must be KT_CKPT8_INT8 or KT_CKPT8_E4M3");
  if (rows * cols == 0) return KT_RAWINT4_OK;
  if (!x || !codes || !scales) return set_error(KT_RAWINT4_EINVAL, "x, codes and scales must be non-NULL");
  if (!is_aligned(x, 16) || !is_aligned(codes, 4) || !is_aligned(scales, 4))
    return set_error(KT_RAWINT4_EINVAL, "x must be 16-byte aligned, codes and scales 4-byte aligned");
  return KT_RAWINT4_OK;
}

}  // namespace kt

using namespace kt;

extern "C" {

int kt_ckpt8_pack(const uint16_t* x, int64_t rows, int64_t cols, int32_t format, uint8_t* codes, uint8_t* scales,
                  void* stream) {
  const int rc = check_ckpt8(x, rows, cols, format, codes, scales);
  if (rc) return rc;
  if (rows * cols == 0) return set_error(KT_RAWINT4_OK, "");
  begin_launches();
  launch_ckpt8_pack(x, rows, cols, format, codes, scales, static_cast<hipStream_t>(stream));
  return finish_launches();
}

int kt_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int32_t format,
                    uint16_t* x, void* stream) {
  const int rc = check_ckpt8(x, rows, cols, format, codes, scales);
  if (rc) return rc;
  if (rows * cols == 0) return set_error(KT_RAWINT4_OK, "");
  begin_launches();
  launch_ckpt8_unpack(codes, scales, rows, cols, format, x, static_cast<hipStream_t>(stream));
  return finish_launches();
}

}  // extern "C"
