// Conversions of values to 8 bits that the quantizers share: scales of a block or
// a row from its largest magnitude, and the codes under them.
#pragma once

#include <hip/hip_runtime.h>

#include "qg_device.h"

namespace qg {

// Scale exponent of a block whose largest magnitude has the fp32 pattern amax
// (a bf16 value widened, sign cleared): floor(log2) - 8, clamped at -127; 0
// for an all-zero block.
__device__ __forceinline__ int mx_block_exp(uint32_t amax) {
  if (amax == 0) return 0;
  return max((int)(amax >> 23) - 135, -127);  // subnormal maxima give -127 too
}

// e4m3 codes of two values already divided by the block scale.  The division
// by a power of two is exact for bf16 inputs (fp32 denormals are kept), the
// clamp to +-448 gives the saturation (values in (448, 464) round to 448
// anyway), and v_cvt_pk_fp8_f32 rounds to nearest-even into OCP e4m3; the
// sign survives, so a negative value that rounds to zero becomes 0x80.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  a = __builtin_amdgcn_fmed3f(a, -448.f, 448.f);
  b = __builtin_amdgcn_fmed3f(b, -448.f, 448.f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// largest value over the lane's quad (lanes 4i .. 4i + 3)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));  // [1,0,3,2]
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));  // [2,3,0,1]
  return v;
}

// FP8 with fp32 scales.  The scale of a block with largest magnitude a is
// s = a / 448 (IEEE fp32 division; 1 for an all-zero block) and each element
// becomes e4m3 of the fp32 quotient v / s (IEEE division, then the
// nearest-even e4m3 of e4m3_pair, saturated at 448).
__device__ __forceinline__ float fp8_block_scale(float amax) { return amax > 0.f ? amax / 448.f : 1.f; }

__device__ __forceinline__ uint2 fp8_store8(const float (&v)[8], float s) {
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    c[h] = e4m3_pair(v[4 * h] / s, v[4 * h + 1] / s) | (e4m3_pair(v[4 * h + 2] / s, v[4 * h + 3] / s) << 16);
  return uint2{c[0], c[1]};
}

// scale of a row with largest magnitude `most`; code of v, IEEE division and
// ties to even
__device__ __forceinline__ float i8_scale(float most) { return most > 0.f ? most / 127.f : 1.f; }
__device__ __forceinline__ uint32_t i8_codes4(const float *v, float s) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)rintf(v[i] / s) & 255u) << (8 * i);
  return w;
}
__device__ __forceinline__ void unpack8(const u32x4 &w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// two values rounded to bf16 (nearest-even, a NaN stays a NaN), the first in the low half
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

}  // namespace qg
