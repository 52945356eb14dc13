// Quantization of eight bf16 values at a time, shared by the kernels that read
// bf16 rows themselves (quantizers, small products, the few-token layer).
#pragma once

#include "mx_device.h"

namespace mxk {

typedef short s16x2 __attribute__((ext_vector_type(2)));

// E8M0 byte of an MXFP4 block from the bits of its largest |bf16|.
__device__ __forceinline__ uint32_t e8m0_fp4_from_absbits(uint32_t amax_bits) {
  if (amax_bits >= 0x7F80u) return 0xFFu;
  const int e = (int)(amax_bits >> 7) - 2;
  return (uint32_t)(e > 0 ? e : 0);
}

// Two bf16 values -> two E2M1 codes in byte SEL of `old`; the convert divides
// by `scale` = 2^(byte - 127), given as the float whose exponent field is the
// byte.
template <int SEL>
__device__ __forceinline__ uint32_t cvt2_e2m1(uint32_t old, uint32_t pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, pair), scale, SEL);
}

// 8 bf16 values (4 dwords) of one block -> 8 codes in a dword.
__device__ __forceinline__ uint32_t quant8_fp4(v4i w, uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  uint32_t c = cvt2_e2m1<0>(0u, (uint32_t)w[0], scale);
  c = cvt2_e2m1<1>(c, (uint32_t)w[1], scale);
  c = cvt2_e2m1<2>(c, (uint32_t)w[2], scale);
  c = cvt2_e2m1<3>(c, (uint32_t)w[3], scale);
  return byte == 0xFFu ? 0u : c;
}

// Four packed bf16 pairs of a block with scale byte `byte` -> eight E4M3
// codes.  The convert divides by the scale and rounds to nearest even but does
// not saturate, so magnitudes are clamped to 448 * 2^(byte - 127) first, as
// bf16 bits (1.75 * 2^(byte + 8 - 127): mantissa bits 0x60).
__device__ __forceinline__ v2i quantize8(v4i w, uint32_t byte, uint32_t most) {
  const float scale = __uint_as_float(byte << 23);
  v2i q;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s16x2 r = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t u = (uint32_t)w[2 * i + j];
      const us2 m = __builtin_elementwise_min(__builtin_bit_cast(us2, u & 0x7FFF7FFFu), __builtin_bit_cast(us2, most));
      const uint32_t v = __builtin_bit_cast(uint32_t, m) | (u & 0x80008000u);
      if (j == 0) r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, v), scale, 0);
      else r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, v), scale, 1);
    }
    q[i] = __builtin_bit_cast(int, r);
  }
  return q;
}

// Largest |bf16| bits of eight values, as a packed pair still to be combined.
__device__ __forceinline__ us2 absmax8x2(v4i w) {
  us2 m = __builtin_bit_cast(us2, (uint32_t)w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, (uint32_t)w[i] & 0x7FFF7FFFu));
  return m;
}

}  // namespace mxk
