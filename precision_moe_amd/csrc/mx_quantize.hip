// Microscaled quantization, the way back, and the activation between two
// products with its 8-bit checkpoint. All are bound by memory: one pass, every
// value read once and written once. A lane holds 8 consecutive elements, four
// lanes a block of 32, whose largest magnitude is two quad permutations away.
// Measured, 268M elements: FP32 to E2M1 240 us, E2M1 to BF16 111 to 118 us (5.1 and 5.8 TB/s; a
// plain copy reaches 5.1); up to some hundred KB the calls are launches (2.4 us).
#include "kernels.h"
#include "mx.h"

namespace pmoe {

// ---------------------------------------------------------------- quantize, dequantize
template <bool kF32>
__device__ __forceinline__ void load8(const void* x, long group, float (&v)[8]) {
  if constexpr (kF32) {
    const float4* p = static_cast<const float4*>(x) + 2 * group;
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    unpack8(static_cast<const uint4*>(x)[group], v);
  }
}

// Codes of eight elements of this lane's block (all four lanes call) and, from
// the block's first lane, the scale byte.
template <MxFormat F>
__device__ __forceinline__ void store_block(float (&v)[8], long group, uint8_t* codes, uint8_t* scales) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
  const uint32_t byte = mx_scale_byte<F>(quad_max(m));
  const bool bad = byte == kMxNan;
  if constexpr (F == kE2M1) {
    const uint32_t c = mx_codes8_e2m1(v, mx_scale(byte));
    reinterpret_cast<uint32_t*>(codes)[group] = bad ? 0u : c;
  } else {
    const uint2 c = mx_codes8_e4m3(v, byte);
    reinterpret_cast<uint2*>(codes)[group] = make_uint2(bad ? 0u : c.x, bad ? 0u : c.y);
  }
  if ((group & 3) == 0) scales[group >> 2] = (uint8_t)byte;
}

template <bool kF32, MxFormat F>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, long groups,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  // groups is a multiple of 4, so the lanes of a block stay together
  for (long g = blockIdx.x * 256L + threadIdx.x; g < groups; g += gridDim.x * 256L) {
    float v[8];
    load8<kF32>(x, g, v);
    store_block<F>(v, g, codes, scales);
  }
}

template <bool kF32, MxFormat F>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, long groups,
                                                            void* __restrict__ out) {
  for (long g = blockIdx.x * 256L + threadIdx.x; g < groups; g += gridDim.x * 256L) {
    float v[8];
    if constexpr (F == kE2M1)
      mx_values8(reinterpret_cast<const uint32_t*>(codes)[g], scales[g >> 2], v);
    else
      mx_values8(reinterpret_cast<const uint2*>(codes)[g], scales[g >> 2], v);
    if constexpr (kF32) {
      float4* o = static_cast<float4*>(out) + 2 * g;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      static_cast<uint4*>(out)[g] = pack8(v);
    }
  }
}

static int group_grid(long groups) {
  const long g = (groups + 255) / 256;
  return (int)(g < 1 << 20 ? g : 1 << 20);
}

template <bool kF32, MxFormat F>
static void quantize(const void* x, long groups, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  mx_quantize_kernel<kF32, F><<<group_grid(groups), 256, 0, s>>>(x, groups, codes, scales);
}

hipError_t launch_mx_quantize(const void* x, bool f32, bool e4m3, long n, uint8_t* codes, uint8_t* scales,
                              hipStream_t s) {
  if (f32)
    e4m3 ? quantize<true, kE4M3>(x, n / 8, codes, scales, s) : quantize<true, kE2M1>(x, n / 8, codes, scales, s);
  else
    e4m3 ? quantize<false, kE4M3>(x, n / 8, codes, scales, s) : quantize<false, kE2M1>(x, n / 8, codes, scales, s);
  return hipGetLastError();
}

template <bool kF32, MxFormat F>
static void dequantize(const uint8_t* codes, const uint8_t* scales, long groups, void* out, hipStream_t s) {
  mx_dequantize_kernel<kF32, F><<<group_grid(groups), 256, 0, s>>>(codes, scales, groups, out);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, bool e4m3, long n, bool f32, void* out,
                                hipStream_t s) {
  if (f32)
    e4m3 ? dequantize<true, kE4M3>(codes, scales, n / 8, out, s) : dequantize<true, kE2M1>(codes, scales, n / 8, out, s);
  else
    e4m3 ? dequantize<false, kE4M3>(codes, scales, n / 8, out, s)
         : dequantize<false, kE2M1>(codes, scales, n / 8, out, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------- activation
// Clamp of the gate from above and of up on both sides; comparisons that a NaN fails keep it.
__device__ __forceinline__ float clamp_gate(float g, float L) { return L > 0.0f && g > L ? L : g; }
__device__ __forceinline__ float clamp_up(float u, float L) {
  return L > 0.0f ? (u > L ? L : (u < -L ? -L : u)) : u;
}

constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0c0p-26f;  // log2(e) = kHi + kLo

// exp(-g) in FP32 within 3 units in the last place for -87 <= g <= 100 (above: that of
// 100, which vanishes beside 1): the product with log2(e) is carried in two parts, as
// its rounding alone would cost |g| units.
__device__ __forceinline__ float exp_neg(float g) {
  g = g > 100.0f ? 100.0f : g;
  const float t = -g * kHi;
  const float r = __builtin_fmaf(-g, kHi, -t) - g * kLo;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * 0x1.62e430p-1f, e);
}

// h = silu(g) * u of eight elements, quantized to E2M1. The stored codes are
// those of the activation itself, not of its FP32 rounding: FP32 arithmetic is
// within kNear of h, so where h * (1 - kNear) and h * (1 + kNear) get the same
// code, and the block's amax the same exponent, the code is decided; else (some
// 1 in 3000 blocks, and values near the ends of FP32's range) the block is
// computed again in FP64. Without this, an element next to a border would move
// by a whole step of 4 bits with the last bit of the exponential.
constexpr float kNear = 0x1p-19f;  // 32 units of 2^-24: about four times the FP32 error

__device__ __forceinline__ uint32_t e2m1_code(double a) {
  return (uint32_t)(a > 0.25) + (uint32_t)(a >= 0.75) + (uint32_t)(a > 1.25) + (uint32_t)(a >= 1.75) +
         (uint32_t)(a > 2.5) + (uint32_t)(a >= 3.5) + (uint32_t)(a > 5.0);
}

__device__ __forceinline__ void swiglu_block_exact(const float (&g)[8], const float (&u)[8], uint32_t& codes,
                                                uint32_t& byte) {
  double h[8];
  double m = 0.0;
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = (double)g[i] / (1.0 + exp(-(double)g[i])) * (double)u[i];
    if (magnitude((float)h[i]) >= 0x7F800000u) bad = 1;  // beyond FP32's largest, or NaN
    m = fmax(m, fabs(h[i]));
  }
  m = fmax(m, __shfl_xor(m, 1, 64));
  m = fmax(m, __shfl_xor(m, 2, 64));
  if (quad_max(bad)) {
    byte = kMxNan;
    codes = 0;
    return;
  }
  const int e = (int)((__double_as_longlong(m) >> 52) & 0x7FF) - 1023 + 127 - (int)kMxEmax<kE2M1>;
  byte = m > 0.0 && e > 0 ? (uint32_t)e : 0u;
  const double inv = __longlong_as_double((long long)(1023 + 127 - (int)byte) << 52);
  codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t sign = (uint32_t)((unsigned long long)__double_as_longlong(h[i]) >> 63);
    codes |= (e2m1_code(fabs(h[i] * inv)) | sign << 3) << (4 * i);
  }
}

__device__ __forceinline__ void swiglu_block(float (&g)[8], float (&u)[8], float L, uint32_t& codes, uint32_t& byte) {
  float h[8];
  uint32_t m = 0;
  bool far = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = clamp_gate(g[i], L);
    u[i] = clamp_up(u[i], L);
    h[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + exp_neg(g[i])) * u[i];
    m = max(m, magnitude(h[i]));
    far |= !(g[i] >= -80.0f);  // the exponential nears FP32's end, or a NaN
  }
  m = quad_max(m);
  const float amax = __uint_as_float(m);
  const uint32_t lo = mx_scale_byte<kE2M1>(__float_as_uint(amax * (1.0f - kNear)));
  byte = mx_scale_byte<kE2M1>(__float_as_uint(amax * (1.0f + kNear)));
  bool again = far | (lo != byte) | (m >= 0x7F000000u) | (m != 0 && m < 0x0D800000u);  // outside [2^-100, 2^127)
  const float s = mx_scale(byte);
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = h[i] * (1.0f - kNear);
    b[i] = h[i] * (1.0f + kNear);
  }
  codes = mx_codes8_e2m1(a, s);
  again |= codes != mx_codes8_e2m1(b, s);
  if (quad_max(again)) swiglu_block_exact(g, u, codes, byte);
}

__device__ __forceinline__ long counted_rows(const int* row_count, long R) {
  if (!row_count) return R;
  const long n = *row_count;
  return n < 0 ? 0 : (n < R ? n : R);
}

// Forward. A lane takes group c (8 elements) of row r: gate and up of the same
// outputs, so that h, its block and both blocks of the checkpoint stay in four lanes.
// 32763 rows, I = 2048, with the checkpoint: 100 to 118 us for 444 MB (the rate of a copy: 87),
// the vector instructions of the exponential, the two codings and the check of the exact value near
// their limit; a fifth fewer of them did not shorten a forward and backward call (218 us). Four
// groups a lane in flight took longer (6.5 instead of 3.5 us at 96 rows). 96 rows: 3.5 to 4.2 us.
template <bool kSwiglu, bool kKeep>
__global__ __launch_bounds__(256) void mx_activation_kernel(const uint16_t* __restrict__ y, long R, int I, float L,
                                                            const int* __restrict__ row_count,
                                                            uint8_t* __restrict__ hq, uint8_t* __restrict__ h_sf,
                                                            uint8_t* __restrict__ y8, uint8_t* __restrict__ y8_sf) {
  const int per = I / 8;  // groups of a row of h, a multiple of 4
  const long total = counted_rows(row_count, R) * per;
  for (long i = blockIdx.x * 256L + threadIdx.x; i < total; i += gridDim.x * 256L) {
    const long r = i / per;
    const int c = (int)(i - r * per);
    float g[8];
    uint32_t codes, byte;
    if constexpr (kSwiglu) {
      const long ga = r * 2 * per + c, ua = ga + per;  // groups of the gate and of up in y
      float u[8];
      load8<false>(y, ga, g);
      load8<false>(y, ua, u);
      if constexpr (kKeep) {
        float t[8], w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = g[k], w[k] = u[k];
        store_block<kE4M3>(t, ga, y8, y8_sf);
        store_block<kE4M3>(w, ua, y8, y8_sf);
      }
      swiglu_block(g, u, L, codes, byte);
      reinterpret_cast<uint32_t*>(hq)[i] = codes;
      if ((c & 3) == 0) h_sf[i >> 2] = (uint8_t)byte;
    } else {
      load8<false>(y, i, g);
      if constexpr (kKeep) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = g[k];
        store_block<kE4M3>(t, i, y8, y8_sf);
      }
      // exact in FP32: the square of 8 significant bits
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = g[k] < 0.0f ? 0.0f : g[k] * g[k];
      store_block<kE2M1>(g, i, hq, h_sf);
    }
  }
}

// Both gradients of SwiGLU at a gate below kLowGate, where s = exp(gate) = m 2^n, 1/2 <= m <= 1, beside
// 1: s alone is below FP32's normal numbers, its product with d h and up need not be, so the power of two
// is applied to that. What a subnormal loses then is at most 2^-150, times a gate of at most 1000, below
// half of BF16's smallest step (2^-134). Below -1000 both gradients are 0 whatever the other factors are.
constexpr float kLowGate = -87.0f;
__device__ __forceinline__ void swiglu_grad_low(float d, float g, float u, float& dg, float& du) {
  g = g < -1000.0f ? -1000.0f : g;
  const float n = __builtin_ceilf(g * kHi);
  const float m = __builtin_amdgcn_exp2f(__builtin_fmaf(g, kHi, -n) + g * kLo);
  dg = __builtin_amdgcn_ldexpf(d * u * m, (int)n) * (1.0f + g);
  du = __builtin_amdgcn_ldexpf(d * m, (int)n) * g;
}

// Backward from the checkpoint: with y the values that it stands for,
//   squared ReLU  d y = 2 max(y, 0) d h
//   SwiGLU        d gate = d h * up * s (1 + gate (1 - s)),  d up = d h * gate * s,  s = 1 / (1 + exp(-gate)),
// gate and up clamped, and no gradient through what the clamp cut off. 32763 rows, I = 2048:
// 95 us for 541 MB, 5.7 TB/s, more than a plain copy's 5.1; the vector units are busy throughout too.
template <bool kSwiglu>
__global__ __launch_bounds__(256) void mx_activation_backward_kernel(
    const uint16_t* __restrict__ dh, const uint8_t* __restrict__ y8, const uint8_t* __restrict__ y8_sf, long R, int I,
    float L, const int* __restrict__ row_count, uint16_t* __restrict__ dy) {
  const int per = I / 8;
  const long total = counted_rows(row_count, R) * per;
  for (long i = blockIdx.x * 256L + threadIdx.x; i < total; i += gridDim.x * 256L) {
    const long r = i / per;
    const int c = (int)(i - r * per);
    float d[8], g[8];
    load8<false>(dh, i, d);
    const uint2* codes = reinterpret_cast<const uint2*>(y8);
    if constexpr (kSwiglu) {
      const long ga = r * 2 * per + c, ua = ga + per;
      float u[8], dg[8], du[8];
      bool low = false;
      mx_values8(codes[ga], y8_sf[ga >> 2], g);
      mx_values8(codes[ua], y8_sf[ua >> 2], u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float gc = clamp_gate(g[k], L), uc = clamp_up(u[k], L);
        const float s = __builtin_amdgcn_rcpf(1.0f + exp_neg(gc));
        const float a = d[k] * uc * (s * __builtin_fmaf(gc, 1.0f - s, 1.0f)), b = d[k] * (gc * s);
        dg[k] = gc != g[k] && g[k] == g[k] ? 0.0f : a;
        du[k] = uc != u[k] && u[k] == u[k] ? 0.0f : b;
        low |= gc < kLowGate;
      }
      if (low) {  // a sigmoid of less than FP32's smallest normal: hardly ever
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!(g[k] < kLowGate)) continue;  // such a gate is not clamped
          const float uc = clamp_up(u[k], L);
          float a, b;
          swiglu_grad_low(d[k], g[k], uc, a, b);
          dg[k] = a;
          du[k] = uc != u[k] && u[k] == u[k] ? 0.0f : b;
        }
      }
      reinterpret_cast<uint4*>(dy)[ga] = pack8(dg);
      reinterpret_cast<uint4*>(dy)[ua] = pack8(du);
    } else {
      mx_values8(codes[i], y8_sf[i >> 2], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = 2.0f * ((g[k] < 0.0f ? 0.0f : g[k]) * d[k]);  // 2 y alone may pass FP32's largest
      reinterpret_cast<uint4*>(dy)[i] = pack8(g);
    }
  }
}

hipError_t launch_mx_activation(const MxActivationParams& p, hipStream_t s) {
  const int grid = group_grid(p.R * (p.I / 8));
  const auto* y = static_cast<const uint16_t*>(p.y);
  if (p.swiglu && p.y8)
    mx_activation_kernel<true, true><<<grid, 256, 0, s>>>(y, p.R, p.I, p.limit, p.row_count, p.hq, p.h_sf, p.y8, p.y8_sf);
  else if (p.swiglu)
    mx_activation_kernel<true, false><<<grid, 256, 0, s>>>(y, p.R, p.I, p.limit, p.row_count, p.hq, p.h_sf, nullptr, nullptr);
  else if (p.y8)
    mx_activation_kernel<false, true><<<grid, 256, 0, s>>>(y, p.R, p.I, p.limit, p.row_count, p.hq, p.h_sf, p.y8, p.y8_sf);
  else
    mx_activation_kernel<false, false><<<grid, 256, 0, s>>>(y, p.R, p.I, p.limit, p.row_count, p.hq, p.h_sf, nullptr, nullptr);
  return hipGetLastError();
}

hipError_t launch_mx_activation_backward(const MxActivationParams& p, const void* dh, void* dy, hipStream_t s) {
  const int grid = group_grid(p.R * (p.I / 8));
  const auto* d = static_cast<const uint16_t*>(dh);
  if (p.swiglu)
    mx_activation_backward_kernel<true><<<grid, 256, 0, s>>>(d, p.y8, p.y8_sf, p.R, p.I, p.limit, p.row_count,
                                                             static_cast<uint16_t*>(dy));
  else
    mx_activation_backward_kernel<false><<<grid, 256, 0, s>>>(d, p.y8, p.y8_sf, p.R, p.I, p.limit, p.row_count,
                                                              static_cast<uint16_t*>(dy));
  return hipGetLastError();
}

}  // namespace pmoe
