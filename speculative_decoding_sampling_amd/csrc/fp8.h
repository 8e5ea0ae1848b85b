// 8-bit floats with a power-of-two scale for each run of 128 values: e4m3
// elements (largest value 448) and an e8m0 scale byte (2^(byte - 127)).
#pragma once

#include "common.h"

namespace specv {

constexpr int kFp8Block = 128;
constexpr int kFp8Lanes = kFp8Block / 8;          // 8 values per lane: 16 lanes share a scale
constexpr uint32_t kFp8NanScale = 255u;
constexpr uint32_t kFp8NanBytes = 0x7f7f7f7fu;
constexpr uint32_t kInfBits = 0x7f800000u;

// Largest of a value over each row of 16 lanes, as unsigned integers: on the
// bits of magnitudes this orders as the floats do, with infinities and NaN
// above every finite value.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, false));
  return v;
}

// Scale byte for the bits of a run's largest magnitude: the smallest power of
// two, at least 2^-126, that brings it to at most 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax) {
  if (amax >= kInfBits) return kFp8NanScale;
  if (amax == 0u) return 127u;
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}

// The 8 values of one lane as e4m3 bytes; all 16 lanes of the run call it
// together.  Scaling by the reciprocal power of two is exact but for results
// below the smallest normal float, which the rounding to e4m3 makes zero.
__device__ __forceinline__ uint2 fp8_pack8(const float* v, uint32_t& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  byte = fp8_scale_byte(row16_max_u32(m));
  if (byte == kFp8NanScale) return make_uint2(kFp8NanBytes, kFp8NanBytes);
  const float inv = __uint_as_float((254u - byte) << 23);
  uint2 r;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
  r.x = (uint32_t)lo;
  r.y = (uint32_t)hi;
  return r;
}

// Two floats as bfloat16 words, round to nearest even, a NaN stays one: one
// instruction for both.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float Float2 __attribute__((ext_vector_type(2)));
  typedef __bf16 Bf16x2 __attribute__((ext_vector_type(2)));
  const Float2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, Bf16x2));
}
__device__ __forceinline__ bf16_t bf16_bits(float f) { return (bf16_t)bf16_pair(f, f); }

}  // namespace specv
