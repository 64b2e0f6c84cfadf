// E4M3 with one UE8M0 scale per 128 columns, on vectors of eight columns a
// thread: the scale rule of the SwiGLU epilogue, encoding, decoding, and the
// 16-byte bf16 vectors they come from and go to.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace mg {

// The smallest s with amax <= 448 * 2^(s-127), clamped to [1, 254]; 127 for
// an all-zero block.  amax = 1.m * 2^(E-127) and 448 = 1.75 * 2^8, so
// s = E - 8, plus one when 1.m > 1.75.
__device__ __forceinline__ int32_t ue8m0_of_amax(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int32_t s = (int32_t)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax == 0.0f ? 127 : min(max(s, 1), 254);
}
// 2^(127-s) for s in [1, 254]: the subnormal 2^-127 for s = 254.
__device__ __forceinline__ float ue8m0_inverse(int32_t s) {
  return s < 254 ? __uint_as_float((uint32_t)(254 - s) << 23) : __uint_as_float(0x00400000u);
}
// 2^(s-127): the subnormal 2^-127 for s = 0, NaN for s = 255.
__device__ __forceinline__ float ue8m0_value(uint32_t s) {
  return s == 0 ? __uint_as_float(0x00400000u) : s == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(s << 23);
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Maximum magnitude of a 128-column block held by 16 consecutive lanes, eight
// columns each; NaN elements do not count.
__device__ __forceinline__ float block_amax(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// Nearest E4M3 values of x * inv, ties to even, magnitudes past 448 to 448.
__device__ __forceinline__ uint2 e4m3x8_encode(const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2((h[0] & 0xffffu) | (h[1] << 16), (h[2] & 0xffffu) | (h[3] << 16));
}
// Values code * scale of eight E4M3 codes.
__device__ __forceinline__ void e4m3x8_decode(const uint2& q, float scale, float (&x)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

}  // namespace mg
