// E4M3 with one UE8M0 scale per 128 columns, on vectors of eight columns a
// thread: the scale rule of the SwiGLU epilogue, encoding, decoding, and the
// 16-byte bf16 vectors they come from and go to.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace mg {

// The smallest s in [1, 254] with amax <= 448 * 2^(s-127); 127 for an all-zero
// block.  amax = 1.m * 2^(E-127) and 448 = 1.75 * 2^8, so s = E - 8, plus one
// when 1.m > 1.75: adding 0x1fffff carries into the exponent exactly then.
// E - 8 is at most 247 (an infinity), and amax is not NaN.
__device__ __forceinline__ int32_t ue8m0_of_amax(float amax) {
  const int32_t s = (int32_t)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
  return amax == 0.0f ? 127 : max(s, 1);
}
// 2^(127-s) for s in [1, 253].
__device__ __forceinline__ float ue8m0_inverse(int32_t s) { return __uint_as_float((uint32_t)(254 - s) << 23); }
// 2^(s-127): the subnormal 2^-127 for s = 0, NaN for s = 255.
__device__ __forceinline__ float ue8m0_value(uint32_t s) {
  return s == 0 ? __uint_as_float(0x00400000u) : s == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(s << 23);
}
// The same of the two scales in a word's low half.
__device__ __forceinline__ float2 ue8m0x2_value(uint32_t s) {
  const __nv_bfloat162_raw r = __nv_cvt_e8m0x2_to_bf162raw((__nv_fp8x2_storage_t)s);
  return make_float2(__uint_as_float((uint32_t)r.x << 16), __uint_as_float((uint32_t)r.y << 16));
}

// Two fp32 operations in one instruction (sm_100 and later), each rounded as
// the single ones are.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t bf16x2_to_f32x2(uint32_t w) {
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(uint64_t v) {
  const float2 f = unpack2(v);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));   // NaN: the other operand
  return r;
}
// Largest magnitude among eight bf16 in each half of the word (even columns
// in the low half, odd ones in the high half); NaN does not count.
__device__ __forceinline__ uint32_t bf16x8_amax2(const uint4& v) {
  const uint32_t a = bf16x2_max(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
  const uint32_t b = bf16x2_max(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
  return bf16x2_max(bf16x2_max(a, b), 0u);
}
// The two halves' maxima over a 128-column block held by 16 consecutive lanes.
__device__ __forceinline__ uint32_t block_max2(uint32_t m) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = bf16x2_max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Maximum magnitude of the block of bf16 columns.
__device__ __forceinline__ float block_amax_bf16(const uint4& v) {
  uint32_t m = bf16x8_amax2(v);
  m = block_max2(bf16x2_max(m, m >> 16));     // the high half holds odd columns only: not used
  return bf16_lo(m);
}

// Maximum magnitude of a block of fp32 columns, 16 lanes, eight columns each;
// NaN elements do not count.
__device__ __forceinline__ float block_amax(const uint64_t (&x)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(x[i]);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// Nearest E4M3 values of x * inv, ties to even, magnitudes past 448 to 448.
__device__ __forceinline__ uint2 e4m3x8_encode(const uint64_t (&x)[4], float inv) {
  const uint64_t k = pack2(inv, inv);
  uint32_t h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2(mul2(x[2 * i], k)), b = unpack2(mul2(x[2 * i + 1], k));
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(h[i])
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  }
  return make_uint2(h[0], h[1]);
}
__device__ __forceinline__ void bf16x8_to_f32x2(const uint4& v, uint64_t (&x)[4]) {
  x[0] = bf16x2_to_f32x2(v.x);
  x[1] = bf16x2_to_f32x2(v.y);
  x[2] = bf16x2_to_f32x2(v.z);
  x[3] = bf16x2_to_f32x2(v.w);
}
__device__ __forceinline__ uint4 f32x2_to_bf16x8(const uint64_t (&x)[4]) {
  return make_uint4(f32x2_to_bf16x2(x[0]), f32x2_to_bf16x2(x[1]), f32x2_to_bf16x2(x[2]), f32x2_to_bf16x2(x[3]));
}
// Values code * scale of eight E4M3 codes.
__device__ __forceinline__ void e4m3x8_decode(const uint2& q, float scale, uint64_t (&x)[4]) {
  const uint64_t k = pack2(scale, scale);
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    x[i] = mul2(pack2(f.x, f.y), k);
  }
}

}  // namespace mg
