// act.cuh -- the activations of the fused operators and their derivatives, in fp32.
//
// SiLU and tanh-GELU are both x times the logistic function of 2u (u = x / 2, or
// u = sqrt(2/pi) (x + 0.044715 x^3)), which has no cancellation for negative x the
// way 1 + tanh(u) has.  NaN stays NaN in every one of them.
#pragma once

#include <cuda_runtime.h>

namespace w4 {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;
// Bound of 0.044715 x^2 in tanh-GELU's slope: from |x| of some 10 on it is multiplied by 0 (s is 0
// or 1), which infinity would turn into NaN where x^2 is past fp32.
constexpr float kCubicMax = 1e30f;

// 1 / (1 + exp(-v)); exp overflows to infinity for v < -88, which gives 0 as it should.
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

__device__ __forceinline__ float act_fwd(float x, int act) {
  switch (act) {
    case kActRelu: return x < 0.0f ? 0.0f : x;
    case kActSilu: return x * logistic(x);
    case kActGelu: return 0.5f * x * erfcf(-0.7071067811865476f * x);
    case kActGeluTanh: return x * logistic(2.0f * kSqrt2OverPi * (x + kGeluCubic * x * x * x));
    default: return x;
  }
}

// act of four values, one switch for all of them; GELU's erfc out of line, so that an epilogue
// stays small: inlined for every value of an unrolled loop, the activations were most of
// a kernel's instructions, and its epilogue waited for their way into the caches.
__device__ __noinline__ float gelu_erf(float x) { return 0.5f * x * erfcf(-0.7071067811865476f * x); }
__device__ __forceinline__ void act_fwd4(float (&z)[4], int act) {
  if (act == kActNone) return;
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = z[j] < 0.0f ? 0.0f : z[j];
  } else if (act == kActGelu) {
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      z[0] = gelu_erf(z[0]);  // one call in a loop that turns the four values round
      const float t = z[0];
      z[0] = z[1]; z[1] = z[2]; z[2] = z[3]; z[3] = t;
    }
  } else {
    // x times the logistic function of x, or of 2 sqrt(2/pi) (x + 0.044715 x^3); b x first, so
    // that SiLU's 0 never meets an x^2 past fp32
    const float a = act == kActSilu ? 1.0f : 2.0f * kSqrt2OverPi, b = act == kActSilu ? 0.0f : kGeluCubic;
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] *= logistic(a * fmaf(b * z[j] * z[j], z[j], z[j]));
  }
}

// act(x) and act'(x)
__device__ __forceinline__ void act_both(float x, int act, float &y, float &dy) {
  switch (act) {
    case kActRelu:
      y = x < 0.0f ? 0.0f : x;
      dy = x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);  // NaN stays NaN
      break;
    case kActSilu: {
      const float s = logistic(x);
      y = x * s;
      dy = s + y * (1.0f - s);  // s (1 + x (1 - s)): off by an ulp of x where s is near 1
      break;
    }
    case kActGelu: {
      const float c = 0.5f * erfcf(-0.7071067811865476f * x);
      y = x * c;
      dy = c + x * 0.3989422804014327f * __expf(-0.5f * x * x);
      break;
    }
    case kActGeluTanh: {
      const float v = 2.0f * kSqrt2OverPi * (x + kGeluCubic * x * x * x);
      const float s = logistic(v);
      y = x * s;
      dy = s + y * (1.0f - s) * 2.0f * kSqrt2OverPi * (1.0f + 3.0f * fminf(kGeluCubic * x * x, kCubicMax));
      break;
    }
    default:
      y = x;
      dy = 1.0f;
  }
}

// act and act' of eight values with one switch, small like act_fwd4.  SiLU and tanh-GELU are
// x s with s the logistic function of a (x + b x^3): act' = s + x s (1 - s) a (1 + 3 b x^2).
__device__ __noinline__ float2 gelu_erf_both(float x) {
  const float c = 0.5f * erfcf(-0.7071067811865476f * x);
  return make_float2(x * c, c + x * 0.3989422804014327f * __expf(-0.5f * x * x));
}
__device__ __forceinline__ void act_both8(const float (&x)[8], int act, float (&y)[8], float (&dy)[8]) {
  if (act >= kActSilu && act != kActGelu) {
    const float a = act == kActSilu ? 1.0f : 2.0f * kSqrt2OverPi, b = act == kActSilu ? 0.0f : kGeluCubic;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = fminf(b * x[j] * x[j], kCubicMax);
      const float s = logistic(a * fmaf(q, x[j], x[j]));
      y[j] = x[j] * s;
      dy[j] = fmaf(y[j] * (1.0f - s), a * fmaf(3.0f, q, 1.0f), s);
    }
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 r = gelu_erf_both(x[j]);
      y[j] = r.x;
      dy[j] = r.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool cut = act == kActRelu && x[j] <= 0.0f;  // NaN stays NaN
      y[j] = cut ? 0.0f : x[j];
      dy[j] = cut ? 0.0f : act == kActRelu && x[j] != x[j] ? x[j] : 1.0f;
    }
  }
}

// 16- and 32-bit elements by w4_dtype number (0 fp32, 1 fp16, 2 bf16)
__device__ __forceinline__ float load_as_float(const void *p, int dtype, int64_t i) {
  if (dtype == 0) return static_cast<const float *>(p)[i];
  if (dtype == 1) return __half2float(static_cast<const __half *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_from_float(void *p, int dtype, int64_t i, float v) {
  if (dtype == 0) static_cast<float *>(p)[i] = v;
  else if (dtype == 1) static_cast<__half *>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace w4
