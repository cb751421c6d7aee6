// Activations and their gradients for the experts' own products.
#pragma once

#include "device_common.h"

namespace moe {

// no activation: the product itself (value matches MOE_ACT_NONE)
constexpr int kActNone = -1;
// columns of the product before the activation, per output column
constexpr int act_width(int kind) { return kind != kActNone && act_is_gated(kind) ? 2 : 1; }

__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

// Activations whose clamps (fminf, fmaxf) would make a number of a NaN.
__device__ __forceinline__ bool act_clamps(int kind, float limit) {
  return kind == kActRelu2NoMul || kind == kActSwigluOai || kind == kActSwigluStep ||
         (kind == kActSilu && limit > 0.0f);
}
// apply_act for callers' own rows: NaN in the gate or up column gives NaN, so that a row
// that went wrong shows.  kind and limit are uniform: a scalar branch where none clamps.
__device__ __forceinline__ float expert_act(int kind, float g, float u, float limit) {
  const float f = apply_act(kind, g, u, limit);
  return act_clamps(kind, limit) && __builtin_isunordered(g, u) ? g + u : f;
}

// Past kFar a sigmoid is 0 or 1 in fp32 and its slope 0.  What multiplies that 0 is taken
// from kFar: an infinity, or a square that passes fp32's range, would make it NaN.
constexpr float kFar = 256.0f;
__device__ __forceinline__ float from_below(float g) { return g < -kFar ? -kFar : g; }
__device__ __forceinline__ float near_zero(float g) { return g > kFar ? kFar : from_below(g); }

struct ActGrad {
  float gate, up;      // of the gate column (or the only one) and of the up column
};

// The gradient of expert_act at (g, u) for the output's gradient dh, in fp32.
// With f(x) = x s(x), s a sigmoid of slope a at 0 times 4: f' = s + a f (1 - s).
// A clamped value passes its gradient up to and at the limit, none past it.  NaN gives
// NaN, at a clamp too.
__device__ __forceinline__ ActGrad act_grad(int kind, float g, float u, float limit, float dh) {
  if (act_clamps(kind, limit) && __builtin_isunordered(g, u)) return ActGrad{g + u, g + u};
  switch (kind) {
    case kActNone:
      return ActGrad{dh, 0.0f};
    case kActSwigluOai: {
      const float gc = fminf(g, limit), uc = fminf(fmaxf(u, -limit), limit);
      const float s = sigmoid_f32(kSwigluOaiAlpha * gc), f = from_below(gc) * s;
      const float df = s + kSwigluOaiAlpha * near_zero(gc) * s * (1.0f - s);
      return ActGrad{g <= limit ? dh * (uc + 1.0f) * df : 0.0f,
                     fabsf(u) <= limit ? dh * f : 0.0f};
    }
    case kActSwigluStep: {
      const float uc = fminf(fmaxf(u, -limit), limit);
      const float s = sigmoid_f32(g), f = from_below(g) * s;
      return ActGrad{f <= limit ? dh * uc * (s + near_zero(g) * s * (1.0f - s)) : 0.0f,
                     fabsf(u) <= limit ? dh * fminf(f, limit) : 0.0f};
    }
    case kActGelu:
    case kActGeluNoMul: {
      const float phi = 0.5f * erfcf(-g * 0.70710678118654752f), x = near_zero(g);
      const float df = phi + x * 0.39894228040143268f * __expf(-0.5f * x * x);
      return kind == kActGelu ? ActGrad{dh * u * df, dh * from_below(g) * phi}
                              : ActGrad{dh * df, 0.0f};
    }
    case kActGeluTanh:
    case kActGeluTanhNoMul: {
      // (1 + tanh y) / 2 = sigmoid(2y); d(2y)/dg = 2 sqrt(2/pi) (1 + 3 * 0.044715 g^2)
      const float x = near_zero(g), x2 = x * x;
      const float s = sigmoid_f32(1.5957691216057308f * (x + 0.044715f * x2 * x));
      const float df =
          s + x * s * (1.0f - s) * (1.5957691216057308f * (1.0f + 0.134145f * x2));
      return kind == kActGeluTanh ? ActGrad{dh * u * df, dh * (from_below(g) * s)}
                                  : ActGrad{dh * df, 0.0f};
    }
    case kActRelu2NoMul:
      return ActGrad{dh * 2.0f * fmaxf(g, 0.0f), 0.0f};
    default: {                                  // SiLU, gated or not
      const bool gated = kind == kActSilu, clamped = gated && limit > 0.0f;
      const float gc = clamped ? fminf(g, limit) : g;
      const float uc = clamped ? fminf(fmaxf(u, -limit), limit) : u;
      const float s = sigmoid_f32(gc), f = from_below(gc) * s;
      const float df = s + near_zero(gc) * s * (1.0f - s);
      if (!gated) return ActGrad{dh * df, 0.0f};
      return ActGrad{clamped && g > limit ? 0.0f : dh * uc * df,
                     clamped && fabsf(u) > limit ? 0.0f : dh * f};
    }
  }
}

}  // namespace moe
