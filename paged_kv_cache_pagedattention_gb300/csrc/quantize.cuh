// Quantisation of cache elements, shared by the kernels that write the paged cache.
#pragma once

#include "pa_common.cuh"

namespace pa {

// x / scale in IEEE fp32 (correctly rounded division), then FP8 (e4m3 or e5m2)
// round-to-nearest-even with saturation to the largest finite value, via the CUDA
// conversion intrinsic.
template <int CDT>
__device__ __forceinline__ uint8_t quant_fp8(float x, float scale) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE,
                                                    CDT == PA_FP8_E5M2 ? __NV_E5M2 : __NV_E4M3));
}

// The codes of two values, a's in the low byte.
template <int CDT>
__device__ __forceinline__ uint16_t quant_fp8x2(float a, float b, float scale) {
  return __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)), __NV_SATFINITE,
                                  CDT == PA_FP8_E5M2 ? __NV_E5M2 : __NV_E4M3);
}

// E2M1 code of y: round to nearest with ties to the even code, saturating at 6,
// sign kept.  The magnitude code counts the midpoints between neighbouring E2M1
// magnitudes (0, 0.5, 1, 1.5, 2, 3, 4, 6) that |y| lies above; at a midpoint the
// comparison is strict or not so that the tie lands on the even code.
__device__ __forceinline__ uint32_t e2m1_code(float y) {
  const float a = fabsf(y);
  const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                     (a > 5.0f);
  return c | (signbit(y) ? 8u : 0u);
}

// NVFP4 quantisation of one group of 16 elements with fp32 scale s: block
// scale code e4m3(amax / (6 s)), codes e2m1(x / (s b)) packed low nibble first;
// zero codes when the block scale is zero.
__device__ __forceinline__ void quant_nvfp4(const float (&x)[16], float s, uint2& codes, uint8_t& scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  const float q = __fdiv_rn(amax, __fmul_rn(6.0f, s));
  scale = static_cast<uint8_t>(__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3));
  const float b = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(scale), __NV_E4M3)));
  uint32_t w[2] = {0u, 0u};
  if (b != 0.f) {
    const float den = __fmul_rn(s, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 3] |= e2m1_code(__fdiv_rn(x[i], den)) << (4 * (i & 7));
  }
  codes = make_uint2(w[0], w[1]);
}

}  // namespace pa
