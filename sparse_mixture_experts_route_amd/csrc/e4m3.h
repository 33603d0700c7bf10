// The 8-bit row format on the device: blocks of 128 values share a scale 2^e,
// e the smallest integer with max|v| <= 448 * 2^e (448 is the largest e4m3
// value), kept in [-120, 120] and held as the byte e + 127.
#pragma once

#include "common.h"

namespace moe {

constexpr int kQBlock = 128;  // values per scale

template <int V>
struct IntC {
  static constexpr int value = V;
};

__host__ __device__ __forceinline__ int64_t code_pitch(int64_t K) { return (K + 127) / 128 * 128; }
__host__ __device__ __forceinline__ int64_t scale_pitch(int64_t K) { return (K + 2047) / 2048 * 16; }

// The scale byte of a block whose largest magnitude is amax >= 0. 448 is
// 1.75 * 2^8: with amax = 1.f * 2^q, e = q - 8 when .f <= .75 and q - 7 above,
// which the added 0x1FFFFF (one less than .25 of a mantissa) carries into the
// exponent field. Infinities clamp to the largest scale.
__device__ __forceinline__ int scale_byte(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 135;
  return min(max(e, -120), 120) + 127;
}

// 2^-e of a scale byte (a normal float32 for every e kept)
__device__ __forceinline__ float inv_scale(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Four values times inv (exact: a power of two) to four e4m3 codes, round to
// nearest even; what exceeds 464, infinities and NaN become NaN codes.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
  return (uint32_t)r;
}

// A value of another lane of the DPP row (CTRL: a DPP control); every lane of
// the row must be active.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// Largest value over the 16 lanes of a DPP row (rotations by 8, 4, 2 and 1).
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp<0x128>(v));
  v = fmaxf(v, dpp<0x124>(v));
  v = fmaxf(v, dpp<0x122>(v));
  return fmaxf(v, dpp<0x121>(v));
}

}  // namespace moe
