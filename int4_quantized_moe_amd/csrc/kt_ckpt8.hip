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

template <int FMT>
__device__ __forceinline__ float ckpt8_value(uint32_t code) {
  if (FMT == KT_CKPT8_INT8) return (float)(int8_t)code;
  return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

// The scale a byte stands for; NaN for 255.
__device__ __forceinline__ float ckpt8_mult(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : pow2f(byte - 127);
}

// Any column count: half a wave per group, one value per lane.
template <int FMT>
__global__ __launch_bounds__(256) void k_ckpt8_pack(const uint16_t* __restrict__ x, int64_t rows, int64_t cols,
                                                    int64_t ng, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales) {
  const int64_t total = rows * ng;
  const int lane = threadIdx.x & 31;
  for (int64_t g = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); g < total; g += (int64_t)gridDim.x * 8) {
    const int64_t row = g / ng, c = (g - row * ng) * 32 + lane;
    const bool in = c < cols;
    const uint32_t bits = in ? (uint32_t)x[row * cols + c] << 16 : 0u;
    uint32_t a = bits & 0x7fffffffu;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, off));
    const int s = ckpt8_scale<FMT>(a);
    const uint32_t code = s == 255 ? 0u : ckpt8_code<FMT>(__uint_as_float(bits), pow2f(127 - s), ckpt8_limit<FMT>(s));
    if (in) codes[row * cols + c] = (uint8_t)code;
    if (lane == 0) scales[g] = (uint8_t)s;
  }
}

template <int FMT>
__global__ __launch_bounds__(256) void k_ckpt8_unpack(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, int64_t rows, int64_t cols,
                                                      int64_t ng, uint16_t* __restrict__ x) {
  const int64_t total = rows * ng;
  const int lane = threadIdx.x & 31;
  for (int64_t g = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); g < total; g += (int64_t)gridDim.x * 8) {
    const int64_t row = g / ng, c = (g - row * ng) * 32 + lane;
    if (c < cols) x[row * cols + c] = float_to_bf16(ckpt8_value<FMT>(codes[row * cols + c]) * ckpt8_mult(scales[g]));
  }
}

static unsigned group_blocks(int64_t groups) {
  const int64_t b = (groups + 7) / 8;
  return (unsigned)(b < 65536 ? b : 65536);
}

static void launch_ckpt8_pack(const uint16_t* x, int64_t rows, int64_t cols, int format, uint8_t* codes,
                              uint8_t* scales, hipStream_t st) {
  const int64_t ng = (cols + 31) / 32;
  if (rows * ng == 0) return;
  if (format == KT_CKPT8_INT8)
    k_ckpt8_pack<KT_CKPT8_INT8><<<group_blocks(rows * ng), 256, 0, st>>>(x, rows, cols, ng, codes, scales);
  else
    k_ckpt8_pack<KT_CKPT8_E4M3><<<group_blocks(rows * ng), 256, 0, st>>>(x, rows, cols, ng, codes, scales);
  note_launch();
}

void launch_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int format,
                         uint16_t* x, hipStream_t st) {
  const int64_t ng = (cols + 31) / 32;
  if (rows * ng == 0) return;
  if (format == KT_CKPT8_INT8)
    k_ckpt8_unpack<KT_CKPT8_INT8><<<group_blocks(rows * ng), 256, 0, st>>>(codes, scales, rows, cols, ng, x);
  else
    k_ckpt8_unpack<KT_CKPT8_E4M3><<<group_blocks(rows * ng), 256, 0, st>>>(codes, scales, rows, cols, ng, x);
  note_launch();
}

static int check_ckpt8(const void* x, int64_t rows, int64_t cols, int32_t format, const void* codes,
                       const void* scales) {
  if (rows < 0 || cols < 0 || (cols > 0 && rows >= ((int64_t)1 << 40) / cols))
    return set_error(KT_RAWINT4_EINVAL, "rows and cols must be non-negative and rows * cols below 2^40");
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
  begin_launches();
  launch_ckpt8_pack(x, rows, cols, format, codes, scales, static_cast<hipStream_t>(stream));
  return finish_launches();
}

int kt_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int32_t format,
                    uint16_t* x, void* stream) {
  const int rc = check_ckpt8(x, rows, cols, format, codes, scales);
  if (rc) return rc;
  begin_launches();
  launch_ckpt8_unpack(codes, scales, rows, cols, format, x, static_cast<hipStream_t>(stream));
  return finish_launches();
}

}  // extern "C"
