// Device-side building blocks of the microscaled (MX) formats: 32 consecutive
// elements share one power of two X = 2^(b - 127), stored as the byte b (E8M0,
// 255 = NaN), with
//   b = max(floor(log2 amax) + 127 - emax, 0),  element = RNE(x / X), saturating,
// where emax is the exponent of the format's largest value: 2 for E2M1 (6 =
// 1.5 * 2^2), 8 for E4M3 (448 = 1.75 * 2^8). Both conversions run on gfx950's
// scaled converts, which apply the exponent of their FP32 scale operand only;
// the operand (b << 23) therefore works for every b, 0 included (checked on the
// device against the definition, ties included). A block that holds an infinity or a NaN gets b = 255 and zero
// codes: every element of it reads back as NaN.
#pragma once

#include "device.h"

namespace pmoe {

constexpr int kMxBlock = 32;  // elements per E8M0 scale
constexpr uint32_t kMxNan = 255;

enum MxFormat { kE2M1 = 0, kE4M3 = 1 };
template <MxFormat F>
constexpr uint32_t kMxEmax = F == kE2M1 ? 2 : 8;

typedef short shortx2 __attribute__((ext_vector_type(2)));

// Scale byte of a block from the bits of its largest magnitude (sign cleared).
// Subnormal amax has exponent bits 0 and gives byte 0, like every amax below 2^(emax - 126).
template <MxFormat F>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (e == 255) return kMxNan;
  return e > kMxEmax<F> ? e - kMxEmax<F> : 0u;
}

// The maximum of the bits of magnitudes over the 4 lanes that hold a block
// (lanes 4k .. 4k+3): two quad permutations.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return v > b ? v : b;
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Eight elements -> E2M1 codes, element i in nibble i.
__device__ __forceinline__ uint32_t mx_codes8_e2m1(const float (&x)[8], float scale) {
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[2], x[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[6], x[7], scale, 3);
}
// Eight finite elements -> E4M3 codes, element i in byte i. This convert gives NaN
// beyond 464 where the one to E2M1 saturates, and loses subnormal inputs, so the
// elements are divided by X (exactly) and cut at 448 before it.
__device__ __forceinline__ uint2 mx_codes8_e4m3(const float (&v)[8], uint32_t byte) {
  const float inv = __uint_as_float((254u - byte) << 23);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_fmed3f(v[i] * inv, -448.0f, 448.0f);
  shortx2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, x[0], x[1], 1.0f, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, x[2], x[3], 1.0f, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, x[4], x[5], 1.0f, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, x[6], x[7], 1.0f, true);
  return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes -> their values in FP32.
__device__ __forceinline__ void mx_values8(uint32_t codes, uint32_t byte, float (&x)[8]) {
  const float s = mx_scale(byte);
  const float2v_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0);
  const float2v_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1);
  const float2v_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 2);
  const float2v_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 3);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1], x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}
__device__ __forceinline__ void mx_values8(uint2 codes, uint32_t byte, float (&x)[8]) {
  const float s = mx_scale(byte);
  const float2v_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes.x, s, false);
  const float2v_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes.x, s, true);
  const float2v_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes.y, s, false);
  const float2v_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes.y, s, true);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1], x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}

// 16 bytes of BF16 <-> eight FP32 values.
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                    f32x2_to_bf16x2(x[6], x[7]));
}

}  // namespace pmoe
