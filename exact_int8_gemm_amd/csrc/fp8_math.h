// Element arithmetic of the fp8 (OCP e4m3) block quantizers: codes for
// 8 consecutive values of a block that 16 neighbouring lanes hold together.
//
//   a = max |x| over the block;  s = a / 448 (IEEE fp32 division)
//   code = e4m3(min(max(x / s, -448), 448)), nearest even
//
// x / s is the correctly rounded fp32 quotient.  It is not divided out per
// element: with r = fl(1 / s), Markstein's correction (P. Markstein, IBM
// J. Res. Dev. 34(1), 1990) q' = fl(q + fl(x - q s) r), both steps one fma,
// is applied twice to q = fl(x r); the first brings q within one ulp, the
// second rounds it correctly.  Its remainders are exact while nothing
// underflows: for |x / s| >= 2^-11 (below, every code is 0) a remainder is a
// multiple of 2^-57 s, so s >= 2^-90 suffices; smaller scales divide.  The
// sign of a zero code is not specified (-0 and values that round to 0 may
// give 0x00 or 0x80).
#pragma once

#include "../../include/prism.h"
#include "prism_internal.h"

namespace prism {
namespace fp8 {

constexpr int kBlock = 128;
constexpr float kMax = 448.0f;

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

// Eight consecutive values as fp32 (16-byte aligned source).
__device__ inline void load8(const float* p, float* x) {
  const v4f a = *reinterpret_cast<const v4f*>(p), b = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[4 + e] = b[e];
  }
}
__device__ inline void load8(const _Float16* p, float* x) {
  const v8h a = *reinterpret_cast<const v8h*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)a[e];
}
__device__ inline void load8(const __bf16* p, float* x) {
  const v4i a = *reinterpret_cast<const v4i*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __builtin_bit_cast(float, (uint32_t)a[e] << 16);
    x[2 * e + 1] = __builtin_bit_cast(float, (uint32_t)a[e] & 0xffff0000u);
  }
}

// Largest magnitude as its bit pattern: ordered like the magnitudes, and a
// NaN or infinity (>= 0x7f800000) stays on top.
__device__ inline uint32_t absmax8(const float* x) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
  return m;
}

// Scale of a block from the bits of its absmax: NaN for a block with a
// non-finite value.
__device__ inline float block_scale(uint32_t amax) {
  return amax >= 0x7f800000u ? __builtin_nanf("") : __builtin_bit_cast(float, amax) / kMax;
}

// Codes of eight values as two dwords; all 0 when the scale is 0 or NaN.
__device__ inline v2i codes8(const float* x, float s) {
  if (!(s > 0.0f)) return v2i{0, 0};
  const float r = 1.0f / s;
  float q[8];
  if (s >= 0x1p-90f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float t = x[e] * r;
      t = __builtin_fmaf(__builtin_fmaf(-t, s, x[e]), r, t);
      q[e] = __builtin_fmaf(__builtin_fmaf(-t, s, x[e]), r, t);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = x[e] / s;
  }
  v2i c{0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = __builtin_amdgcn_fmed3f(q[4 * h + e], -kMax, kMax);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    c[h] = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w, true);
  }
  return c;
}

}  // namespace fp8
}  // namespace prism
