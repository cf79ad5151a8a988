// Activations of the FFN epilogues (dense linear with an epilogue, MoE layer),
// in fp32 on values that are rounded to fp16 right after.
//
// Accuracy: the target is an error far under half an fp16 step (2^-11
// relative), at a cost that hides behind the tensor-core mainloop (two
// special-function operations and under ten multiply-adds per value).  The
// exponentials and reciprocals are CUDA's fast intrinsics (relative error of a
// few 2^-23 here).
//   silu       z / (1 + e^-z)
//   gelu_tanh  0.5 z (1 + tanh u) = z / (1 + e^-2u),  u = sqrt(2/pi) (z + 0.044715 z^3)
//   gelu       z Phi(z), Phi the normal distribution function: with u = |z| and
//              t = 1 / (1 + 0.3 u), Phi(-u) = e^(-u^2/2) t P(t).  P, of degree 5, is a
//              least-squares fit (reweighted towards the largest relative error) of
//              erfcx(u / sqrt(2)) / (2 t) over 0 <= u <= 9: relative error 2.1e-6, which
//              the factored exponential carries to the far negative tail (3.6e-6
//              relative in fp32 for |z| < 6, past which fp16 has no value left).
// NaN stays NaN; relu(-0) = 0.
#pragma once

#include <cstdint>

namespace fp8q {

enum Activation : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

__device__ __forceinline__ float act_silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

__device__ __forceinline__ float act_gelu_tanh(float z) {
  // -2u = z (-2 sqrt(2/pi) - 2 sqrt(2/pi) 0.044715 z^2)
  const float s = z * fmaf(-0.0713548162726f, z * z, -1.59576912160573f);
  return __fdividef(z, 1.0f + __expf(s));
}

__device__ __forceinline__ float act_gelu(float z) {
  const float u = fabsf(z);
  const float t = __fdividef(1.0f, fmaf(0.3f, u, 1.0f));
  float p = fmaf(-0.0818373346f, t, 0.230586332f);
  p = fmaf(p, t, -0.0340378628f);
  p = fmaf(p, t, 0.153751159f);
  p = fmaf(p, t, 0.111210456f);
  p = fmaf(p, t, 0.120327727f);
  const float q = p * t * __expf(-0.5f * u * u);   // Phi(-|z|)
  // z > 0: z - z q;  z < 0: z q
  return fmaf(z, z > 0.0f ? -q : q, z > 0.0f ? z : 0.0f);
}

// The activation `act` (uniform over the grid: one branch per call site).
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;
    case kActGelu: return act_gelu(z);
    case kActGeluTanh: return act_gelu_tanh(z);
    case kActSilu: return act_silu(z);
    default: return z;
  }
}

}  // namespace fp8q
