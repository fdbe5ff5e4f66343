// Encoding of a block of values in 8 bits (definitions: f8_quantize.cu), for the kernels
// that quantise, and of an fp32 value as bf16 terms.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace qlora {

// An fp32 value as three bf16 terms, 24 bits in all: what each leaves is exact in fp32.
struct Terms {
  __nv_bfloat16 hi, mid, lo;
};
__device__ __forceinline__ Terms terms_of(float v) {
  Terms t;
  t.hi = __float2bfloat16_rn(v);
  v -= __bfloat162float(t.hi);
  t.mid = __float2bfloat16_rn(v);
  t.lo = __float2bfloat16_rn(v - __bfloat162float(t.mid));
  return t;
}

constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ float block_scale_of(float amax, bool e5m2, bool pow2) {
  const float fmax = e5m2 ? 57344.0f : 448.0f;
  if (!pow2) return fmaxf(__fdiv_rn(amax, fmax), kScaleFloor);
  // F = 1.75 2^8 or 1.75 2^15: with amax = m 2^e (1 <= m < 2) the power is
  // e - 8 (e - 15), one more when m > 1.75.  A subnormal amax lies far below the floor.
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - (e5m2 ? 15 : 8) + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, 1);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// |x| of a finite value, 0 for NaN and infinities
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __int_as_float(0x7f800000) ? a : 0.0f;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  a *= inv;
  b *= inv;
  c *= inv;
  d *= inv;
  a = fmaf(a, 0.0f, a);
  b = fmaf(b, 0.0f, b);
  c = fmaf(c, 0.0f, c);
  d = fmaf(d, 0.0f, d);
  constexpr __nv_fp8_interpretation_t kF = E5M2 ? __NV_E5M2 : __NV_E4M3;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, kF);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, kF);
  return lo | (hi << 16);
}

// The largest finite |value| of N words of two bf16 (or one fp32 each), 0 if there is
// none.  bf16: the packed maximum leaves NaN out by itself; only where an infinity
// is left are the finite ones looked for one by one.
template <typename T, int N>
__device__ __forceinline__ float amax_words(const uint32_t (&w)[N]) {
  float a = 0.0f;
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 m = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < N; ++j)
      m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
    a = fmaxf(__low2float(m), __high2float(m));
    if (a < __int_as_float(0x7f800000)) return a;
    a = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
      a = fmaxf(a, fmaxf(finite_abs(__uint_as_float(w[j] << 16)),
                         finite_abs(__uint_as_float(w[j] & 0xffff0000u))));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) a = fmaxf(a, finite_abs(__uint_as_float(w[j])));
  }
  return a;
}

}  // namespace qlora
