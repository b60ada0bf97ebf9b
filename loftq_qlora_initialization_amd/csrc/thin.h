// What the thin products of one adapted layer and of a pool of adapters share: the matrix cores' product, masked
// operands and the pieces of an fp32 sum.
//
// v_mfma_f32_16x16x32_bf16: lane L supplies A[L%16][8(L/16) + j] and
// B[8(L/16) + j][L%16] (j = 0..7) and receives D[4(L/16) + v][L%16] in element v.
#pragma once

#include "dropout.h"

namespace loftq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 8 values of a masked row, elements e .. e + 7 of the flattening (e % 8 == 0)
__device__ __forceinline__ u32x4 drop8(u32x4 v, uint64_t key, uint64_t e, uint32_t thr) {
  const uint64_t z = key + ((e >> 2) + 1) * kMixGamma, w0 = mix64(z), w1 = mix64(z + kMixGamma);
  v[0] = drop_pair(v[0], w0, 0, thr);
  v[1] = drop_pair(v[1], w0, 2, thr);
  v[2] = drop_pair(v[2], w1, 0, thr);
  v[3] = drop_pair(v[3], w1, 2, thr);
  return v;
}

// x = h0 + h1 + h2 in bf16, each the rounding of what the ones before leave: the three hold 24 bits, so the products
// they enter lose nothing against fp32; an infinity or a NaN is all in the first.
__device__ __forceinline__ void split3(float x, __bf16 (&h)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    h[q] = static_cast<__bf16>(x);
    x = __builtin_isfinite(static_cast<float>(h[q])) ? x - static_cast<float>(h[q]) : 0.f;
  }
}

}  // namespace
}  // namespace loftq
