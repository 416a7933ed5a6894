// act.cuh -- the gated block's activations, their slopes, and 16-bit packing.
//
//   silu       act(g) = g s(g)                   s(p) = 1 / (1 + exp(-p))
//   gelu_tanh  act(g) = g s(2 k (g + 0.044715 g^3)), k = sqrt(2 / pi): the tanh
//              form of GELU, since (1 + tanh(z)) / 2 = s(2 z)
//   relu       act(g) = max(g, 0)
// With p(g) the argument above, act'(g) = s + g p'(g) s (1 - s).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace gb300 {
namespace ops {

enum Act : int32_t { kActSilu = 0, kActGeluTanh = 1, kActRelu = 2 };

// exp(-p) overflows to infinity for very negative p, where s is 0; the
// quotient is then exactly 0.
__device__ __forceinline__ float sigmoid(float p) { return __fdividef(1.0f, 1.0f + __expf(-p)); }

constexpr float kGeluA = 1.5957691216057308f;             // 2 sqrt(2 / pi)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

// __fdividef returns 0 for divisors above 2^126: exactly the limit wanted.
// A gate of -inf would give -inf * 0; the limit of every activation there is
// -0 or 0 in exact arithmetic, but the plain formula gives NaN, and so does
// this.
__device__ __forceinline__ float act_value(int32_t act, float g) {
  if (act == kActRelu) return g > 0.0f ? g : (g != g ? g : 0.0f);
  const float p = act == kActSilu ? g : g * fmaf(kGeluB * g, g, kGeluA);
  return g * sigmoid(p);
}

// act(g) and act'(g).
__device__ __forceinline__ void act_both(int32_t act, float g, float& a, float& da) {
  if (act == kActRelu) {
    a = g > 0.0f ? g : (g != g ? g : 0.0f);
    da = g > 0.0f ? 1.0f : 0.0f;
    return;
  }
  const bool silu = act == kActSilu;
  const float p = silu ? g : g * fmaf(kGeluB * g, g, kGeluA);
  const float s = sigmoid(p);
  a = g * s;
  // From |g| = 64 on, GELU's s is 0 or 1: p' must not overflow there.
  const float c = silu ? g : fminf(fmaxf(g, -64.0f), 64.0f);
  const float dp = silu ? 1.0f : fmaf(3.0f * kGeluB * c, c, kGeluA);
  da = fmaf(c * s * dp, 1.0f - s, s);
}

// Two fp32 values rounded to the nearest 16-bit ones, `lo` in the low half.
__device__ __forceinline__ uint32_t pack16(bool bf16, float lo, float hi) {
  if (bf16) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
  }
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack16(bool bf16, uint32_t v) {
  if (bf16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

__device__ __forceinline__ uint16_t round16(bool bf16, float v) {
  if (bf16) {
    __nv_bfloat16 b = __float2bfloat16_rn(v);
    return *reinterpret_cast<uint16_t*>(&b);
  }
  __half h = __float2half_rn(v);
  return *reinterpret_cast<uint16_t*>(&h);
}

__device__ __forceinline__ float widen16(bool bf16, uint16_t v) {
  if (bf16) return __bfloat162float(*reinterpret_cast<__nv_bfloat16*>(&v));
  return __half2float(*reinterpret_cast<__half*>(&v));
}

}  // namespace ops
}  // namespace gb300
