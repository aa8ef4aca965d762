// act.h -- activations and their derivatives in fp32, shared by the epilogues.
#pragma once

#include "device.h"

namespace miep {

// exp(-g) to fp32 accuracy from the hardware's exp2: the product g * log2(e)
// is carried in two parts, the low one applied to first order.  |g| is capped
// where the sigmoid is 1 (or exp(-g) overflows and it is 0) to fp32.
__device__ __forceinline__ float sigmoid(float g) {
  const float c = -fminf(fmaxf(g, -100.f), 100.f);
  const float hi = c * 1.44269502f;                                   // log2(e), rounded to fp32
  const float lo = fmaf(c, 1.44269502f, -hi) + c * 1.92596299e-8f;    // and its rest
  const float e = __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.693147182f, 1.f);   // infinity stays infinity
  return __builtin_amdgcn_rcpf(1.f + e);
}

// The normal distribution function: that of -|z| as 2 to a polynomial of |z|, to
// 4e-8 (1.6e-8 by the coefficients, the rest its fp32 roundings; exp2 adds an ulp of
// the result, 1 - tail for z > 0 half an ulp, 2^-25: under 1e-7 in all).  Least squares
// with the weight that makes it the error of the result, over 0 .. 6; from there on
// the polynomial falls and the result with it.  A dozen instructions a value, where
// formula 7.1.26 of Abramowitz and Stegun takes 17 and the library's erff several
// times that: an epilogue is not hidden behind its product.
__device__ __forceinline__ float normal_cdf(float z) {
  const float x = fabsf(z);
  float q = fmaf(x, -2.77205049e-6f, 3.86207612e-5f);
  q = fmaf(x, q, -0.000182547636f);
  q = fmaf(x, q, -0.000145870072f);
  q = fmaf(x, q, 0.0070754718f);
  q = fmaf(x, q, -0.0525050275f);
  q = fmaf(x, q, -0.459204912f);
  q = fmaf(x, q, -1.15110576f);
  q = fmaf(x, q, -1.f);
  const float tail = __builtin_amdgcn_exp2f(q);
  return z < 0.f ? tail : 1.f - tail;
}

// gelu's tanh form is z * sigmoid(2u), u = sqrt(2/pi) * (z + 0.044715 z^3).
__device__ __forceinline__ float gelu_tanh_sigmoid(float z) {
  return sigmoid(1.59576912f * fmaf(0.044715f * z * z, z, z));
}

// f(z); kActNone and kActSwiglu (whose two halves a caller joins) give z.
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f || z != z ? z : 0.f;
    case kActSilu: return z * sigmoid(z);
    case kActGelu: return z * normal_cdf(z);
    case kActGeluTanh: return z * gelu_tanh_sigmoid(z);
    default: return z;
  }
}

// f'(z)
__device__ __forceinline__ float activate_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActSilu: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    case kActGelu:                                                    // the distribution function and z times its density
      return fmaf(z * 0.398942280f, __builtin_amdgcn_exp2f(z * z * -0.721347520f), normal_cdf(z));
    case kActGeluTanh: {                                              // (s is 0 or 1 long before 64, where the square could overflow)
      const float s = gelu_tanh_sigmoid(z), c = fminf(fmaxf(z, -64.f), 64.f);
      return z != z ? z : s + c * s * (1.f - s) * (1.59576912f * fmaf(0.134145f * c, c, 1.f));
    }
    default: return 1.f;
  }
}

// 8 bf16 numbers as fp32, and back (rounded).
__device__ __forceinline__ void widen(const v4u& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ v4u narrow(const float (&f)[8]) {
  return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

}  // namespace miep
