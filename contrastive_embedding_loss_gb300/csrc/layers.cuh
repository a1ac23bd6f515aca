// layers.cuh -- device helpers of the head's operators: loads and stores of 8 elements of a
// type, activations and their derivatives, and what follows a matrix product's accumulator.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>
#include <type_traits>

#include "layers.h"
#include "ptx.cuh"

namespace ufc {

__device__ __forceinline__ float bf16_low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_high(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// Two floats to packed bf16, nearest even (a in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint16_t to_bf16(float a) { return static_cast<uint16_t>(pack_bf16(a, 0.f) & 0xFFFFu); }

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  v[0] = bf16_low(q.x), v[1] = bf16_high(q.x), v[2] = bf16_low(q.y), v[3] = bf16_high(q.y);
  v[4] = bf16_low(q.z), v[5] = bf16_high(q.z), v[6] = bf16_low(q.w), v[7] = bf16_high(q.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ uint4 pack8(const float2 (&v)[4]) {
  return make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
}

// Eight consecutive elements as floats (16-byte aligned for the 16- and 32-bit types).
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) { *reinterpret_cast<uint4*>(p) = pack8(v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Two floats to packed e4m3, nearest even, saturating (a in the low byte).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// ---------------------------------------------------------------- activations
// Two elements at a time (packed fp32 arithmetic): the elementwise passes are bound by their
// instructions otherwise, not by HBM.  Exponentials and reciprocals are the hardware's
// approximations (about 2 ulp each), and an exponential's argument x is good to 2^-23 x: far below the
// rounding of the bf16 outputs that use them.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 exp2_2(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float2 rcp2(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
// 1 / (1 + 2^x)
__device__ __forceinline__ float2 logistic2(float2 x) { return rcp2(add2(exp2_2(x), both(1.f))); }
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
// Phi(z), the normal distribution function, and e^(-z^2/2), from one exponential:
// Phi(-|z|) = (a1 t + ... + a6 t^6) e^(-z^2/2), t = 1 / (1 + 0.29 |z|), in the manner of Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26, whose coefficients bound the absolute error
// alone (their tail is 0.2 % off at z = -5, 2 % at -10, while gelu(z) = z Phi(z) is rounded to bf16
// relative to itself).  These are fitted to both: the least maximum (by Lawson's iteration) of the
// error over min(1.2e-4 Phi(-|z|), 4e-8), z from 0 to 14.5, where e^(-z^2/2) ends.  Evaluated in fp32
// within 2.2e-7, and within 1.4e-4 of the value.  The gelu's derivative needs both results.
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2& e) {
  const float2 t = rcp2(fma2(make_float2(fabsf(z.x), fabsf(z.y)), both(0.29f), both(1.f)));
  e = exp2_2(mul2(mul2(z, both(-0.5f * kLog2e)), z));
  float2 q = fma2(t, both(-0.08948110044f), both(0.2872057557f));
  q = fma2(t, q, both(-0.09629647434f));
  q = fma2(t, q, both(0.1814696044f));
  q = fma2(t, q, both(0.1001859829f));
  q = fma2(t, q, both(0.1169161946f));
  const float2 tail = mul2(mul2(t, q), e);  // Phi(-|z|)
  const float2 rest = fma2(tail, both(-1.f), both(1.f));
  return make_float2(z.x < 0.f ? tail.x : rest.x, z.y < 0.f ? tail.y : rest.y);
}
__device__ __forceinline__ float2 gelu_tanh_arg(float2 z) {  // -log2(e) 2 sqrt(2 / pi) (z + 0.044715 z^3)
  return mul2(z, fma2(mul2(z, z), both(-kLog2e * kGeluC * 0.044715f), both(-kLog2e * kGeluC)));
}

template <int ACT>
__device__ __forceinline__ float2 act_of2(float2 z) {
  if constexpr (ACT == kActRelu) return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);  // (a NaN stays one)
  if constexpr (ACT == kActGelu) {
    float2 e;
    return mul2(z, normal_cdf2(z, e));
  }
  if constexpr (ACT == kActGeluTanh) return mul2(z, logistic2(gelu_tanh_arg(z)));
  if constexpr (ACT == kActSilu) return mul2(z, logistic2(mul2(z, both(-kLog2e))));
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  return act_of2<ACT>(make_float2(z, z)).x;
}
// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ void act_grad2(float2 z, float2& a, float2& da) {
  a = z, da = both(1.f);
  if constexpr (ACT == kActRelu) {
    a = act_of2<ACT>(z);
    da = make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
  }
  if constexpr (ACT == kActGelu) {
    float2 e;
    const float2 cdf = normal_cdf2(z, e);
    a = mul2(z, cdf);
    da = fma2(mul2(z, both(0.39894228f)), e, cdf);
  }
  if constexpr (ACT == kActGeluTanh) {
    const float2 s = logistic2(gelu_tanh_arg(z));
    a = mul2(z, s);
    // (the factor of z^2 is 0 long before z^2 overflows)
    const float2 zz = mul2(z, z), z2 = make_float2(fminf(zz.x, 1e30f), fminf(zz.y, 1e30f));
    da = fma2(mul2(a, fma2(s, both(-1.f), both(1.f))), fma2(z2, both(kGeluC * 0.134145f), both(kGeluC)), s);
  }
  if constexpr (ACT == kActSilu) {
    const float2 s = logistic2(mul2(z, both(-kLog2e)));
    a = mul2(z, s);
    da = fma2(a, fma2(s, both(-1.f), both(1.f)), s);
  }
}

// Calls f with a run-time activation (uniform over the grid) as a compile-time constant.
template <int ACT>
using ActC = std::integral_constant<int, ACT>;
template <typename F>
__device__ __forceinline__ void for_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(ActC<kActRelu>{}); break;
    case kActGelu: f(ActC<kActGelu>{}); break;
    case kActGeluTanh: f(ActC<kActGeluTanh>{}); break;
    case kActSilu: f(ActC<kActSilu>{}); break;
    default: f(ActC<kActNone>{}); break;
  }
}

// ---------------------------------------------------------------- after the accumulator
// Eight columns c .. c + 7 (c a multiple of 8, c + 8 <= cols) of one row of a linear product.
template <int ACT>
__device__ __forceinline__ void linear_finish8(const Epilogue& e, int64_t row, int64_t c, float (&z)[8]) {
  if (e.x_scale) {
    const float xs = __ldg(e.x_scale + row);
    float ws[8];
    load8(e.w_scale + c, ws);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] *= xs * ws[j];
  }
  if (e.bias) {
    float b[8];
    if (e.bias_type == kF32)
      load8(static_cast<const float*>(e.bias) + c, b);
    else
      load8(static_cast<const uint16_t*>(e.bias) + c, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += b[j];
  }
  if (e.pre) store8(e.pre + row * e.ldp + c, z);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 y = act_of2<ACT>(make_float2(z[j], z[j + 1]));
    z[j] = y.x, z[j + 1] = y.y;
  }
  if (e.res) {
    float r[8];
    load8(e.res + row * e.ldr + c, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += r[j];
  }
  store8(e.y + row * e.ldy + c, z);
}
// The same columns of the gated block: g and u are the two products.
template <int ACT>
__device__ __forceinline__ void gated_finish8(const Epilogue& e, int64_t row, int64_t c, const float (&g)[8],
                                              const float (&u)[8]) {
  if (e.pre) {
    store8(e.pre + row * e.ldp + c, g);
    store8(e.pre + row * e.ldp + e.cols + c, u);
  }
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 y = mul2(act_of2<ACT>(make_float2(g[j], g[j + 1])), make_float2(u[j], u[j + 1]));
    h[j] = y.x, h[j + 1] = y.y;
  }
  store8(e.y + row * e.ldy + c, h);
}

}  // namespace ufc
