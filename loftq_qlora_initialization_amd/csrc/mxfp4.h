// MXFP4 as the library stores it (OCP Microscaling Formats v1.0: FP4 e2m1 elements, one
// e8m0 scale per 32): a rows x cols matrix in blocks of 32 consecutive columns of a row.
//
// Codes: each row is padded with zeros to whole steps of 256 columns (128 bytes), two
// codes per byte, element 2i in the high nibble.  Code = sign << 3 | magnitude index.
// Scales: one byte per block, 2^(byte - 127), 255 = NaN; stored step by step, the 8
// bytes of row i in step k at (k rows + i) 8, so that the rows of a tile's step are
// one contiguous run.  A step is the K step of the tiled product: 128 bytes of codes
// and 8 scales a row, without a tail.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace loftq {

constexpr int kMxBlock = 32, kMxStep = 256;

inline int64_t mx_steps(int64_t cols) { return (cols + kMxStep - 1) / kMxStep; }

namespace {

// The scale byte of a block whose largest magnitude has the bits `amax` (fp32, sign
// cleared): its exponent less that of 4 (FP4's largest binade), at least 2^-127; NaN
// where the block holds an infinity or a NaN.  The value below is floor(log2 amax) - 2
// + 127 for normal amax; subnormal ones have exponent field 0 and give byte 0.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - byte), the factor that takes a block's values to FP4's range (byte <= 252); 0 for a NaN block
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) {
  return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127)
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : (byte == 0u ? __uint_as_float(0x00400000u)
                                                                   : __uint_as_float(byte << 23));
}

// Eight scaled values into a word of codes.  The conversion instruction rounds to the nearest
// e2m1 value, ties to the even code, and takes larger magnitudes to 6; the scale is applied
// before it, exactly, since the instruction's own scale does not reach 2^-127.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
  uint32_t word = 0;   // the instruction puts its first value into the low nibble
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[1], v[0], 1.f, 0);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[3], v[2], 1.f, 1);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[5], v[4], 1.f, 2);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[7], v[6], 1.f, 3);
  return word;
}

// Eight consecutive values of a row (columns c0 .. c0 + 7 of the padded matrix) into a word of
// codes; the four lanes of a quad hold one block and exchange its largest magnitude by two quad
// permutes.
__device__ __forceinline__ uint32_t mx_encode8(const float (&x)[8], uint32_t& byte) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(x[j]) & 0x7FFFFFFFu;
    amax = b > amax ? b : amax;
  }
  const uint32_t o1 = __builtin_amdgcn_mov_dpp(amax, 0xB1, 0xF, 0xF, true);   // quad_perm 1,0,3,2
  amax = o1 > amax ? o1 : amax;
  const uint32_t o2 = __builtin_amdgcn_mov_dpp(amax, 0x4E, 0xF, 0xF, true);   // quad_perm 2,3,0,1
  amax = o2 > amax ? o2 : amax;
  byte = mx_scale_byte(amax);
  const float inv = mx_inverse_scale(byte);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x[j] * inv;
  return mx_codes8(v);
}
__device__ __forceinline__ float fp4_value(uint32_t code) {
  // magnitude code 0: 0, 1: 0.5, else (1 + m / 2) 2^(e - 1) with e = code >> 1 & 3, m = code & 1
  const uint32_t e = code >> 1 & 3u, m = code & 1u;
  const float mag = e == 0u ? 0.5f * static_cast<float>(m)
                            : __uint_as_float(((126u + e) << 23) | (m << 22));
  return code & 8u ? -mag : mag;
}

}  // namespace
}  // namespace loftq
