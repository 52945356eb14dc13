// The sigmoid of the gated activation, and values of MXFP8 codes.
#pragma once

#include "mx_device.h"

namespace mxk {

typedef float v2f __attribute__((ext_vector_type(2)));

// sigmoid(x) = m, or m * 2^-160 where `far`, and 1 - sigmoid(x) = q, off by some
// 2^-22 of the value over the whole fp32 range.  e^-x = 2^y of y = -x / ln 2 by the
// hardware, with what the product rounds away put back.  From y = 120 on (the one
// is lost beside the power) the power is taken with 2^-160: its reciprocal would be
// subnormal past y = 126, which the hardware makes zero, while silu(-90) * u may be
// any number.  Past |y| = 280 the result is 0 or 1, with nothing to put back.
// The hardware's power and reciprocal are within an ulp each.  In the values made of them
// that is no more than the products around them round: of 418 M codes of gradients 314
// are not those of 64 bits, as with a corrected reciprocal (2 more fma a value, 0 to 1%
// of the time); all in fp32 with correctly rounded divisions, 290.
struct Sigmoid {
  float m, q;
  bool far;
};

__device__ __forceinline__ Sigmoid sigmoid_parts(float x) {
  const float y = x * -1.442695041f;
  const float lo = fmaf(x, -1.925963033e-8f, fmaf(x, -1.442695041f, -y));
  Sigmoid s;
  s.far = y > 120.f;
  float p = __builtin_amdgcn_exp2f(s.far ? y - 160.f : y);
  const float whole = fmaf(p * lo, 0.6931471806f, p);
  p = fabsf(y) < 280.f ? whole : p;
  s.m = __builtin_amdgcn_rcpf((s.far ? 0.f : 1.f) + p);
  s.q = s.far ? 1.f : p * s.m;
  return s;
}

// The same for |x| < 80, where nothing leaves fp32's range.
__device__ __forceinline__ Sigmoid sigmoid_near(float x) {
  const float y = x * -1.442695041f;
  const float lo = fmaf(x, -1.925963033e-8f, fmaf(x, -1.442695041f, -y));
  const float e = __builtin_amdgcn_exp2f(y), p = fmaf(e * lo, 0.6931471806f, e);
  Sigmoid s;
  s.m = __builtin_amdgcn_rcpf(1.f + p);
  s.q = p * s.m;
  s.far = false;
  return s;
}

// a * b where a was computed from s.m.  The 2^-160 is split so that neither factor
// falls below fp32's range where the product does not.
__device__ __forceinline__ float scaled(const Sigmoid& s, float a, float b) {
  return __builtin_ldexpf(a, s.far ? -40 : 0) * __builtin_ldexpf(b, s.far ? -120 : 0);
}

// silu(x) * u
__device__ __forceinline__ float silu_mul(float x, float u) {
  const Sigmoid s = sigmoid_parts(x);
  return scaled(s, x * s.m, u);
}

// The scale of an E8M0 byte as fp32: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_from_e8m0(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x00400000u : byte << 23;
  return __uint_as_float(byte == 0xFFu ? 0x7FC00000u : bits);
}

// Four E4M3 codes of a dword -> their values times `scale`.
__device__ __forceinline__ void values4(uint32_t codes, float scale, float* out) {
  const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  out[0] = a[0] * scale;
  out[1] = a[1] * scale;
  out[2] = b[0] * scale;
  out[3] = b[1] * scale;
}
__device__ __forceinline__ void values8(v2i codes, float scale, float* out) {
  values4((uint32_t)codes[0], scale, out);
  values4((uint32_t)codes[1], scale, out + 4);
}

}  // namespace mxk
