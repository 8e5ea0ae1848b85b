// 4-bit floats with a power-of-two scale for each block of 32 values: e2m1
// codes (0, 0.5, 1, 1.5, 2, 3, 4, 6, sign in bit 3), two to a byte, the first in
// the low half, and an e8m0 scale byte (2^(byte - 127)).
#pragma once

#include "common.h"

namespace specv {

constexpr int kFp4Block = 32;
constexpr int kFp4Lanes = kFp4Block / 8;          // 8 values per lane: 4 lanes share a scale
constexpr uint32_t kFp4NanScale = 255u;

// Scale byte for the bits of a block's largest magnitude: the smallest power
// of two, at least 2^-126, that brings it to at most 6 = 1.5 * 2^2.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kFp4NanScale;
  if (amax == 0u) return 127u;
  const int e = (int)(amax >> 23) - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}

// The 8 values of one lane as codes; the block's 4 lanes call it together.
// Scaling by the reciprocal power of two is exact but for results below the
// smallest normal float, which the rounding to a code makes zero.
__device__ __forceinline__ uint32_t fp4_pack8(const float* v, uint32_t& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, false));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, false));
  byte = fp4_scale_byte(m);
  if (byte == kFp4NanScale) return 0u;
  const float inv = __uint_as_float((254u - byte) << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
  return w;
}

}  // namespace specv
