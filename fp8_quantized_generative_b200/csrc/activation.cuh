// Activations of the FFN epilogues (dense linear with an epilogue, MoE layer),
// in fp32 on values that are rounded to fp16 right after.
//
// Accuracy: the target is an error far under half an fp16 step (2^-11
// relative), at a cost that hides behind the tensor-core mainloop: few special
// functions (ex2.approx, rcp.approx: relative error about 2^-22 each; 16 a cycle and
// SM, so each costs as much as eight multiply-adds) and few multiply-adds.
//   silu       z / (1 + e^-z)
//   gelu_tanh  0.5 z (1 + tanh u) = z / (1 + e^-2u),  u = sqrt(2/pi) (z + 0.044715 z^3)
//              Both: one exponential a value and one reciprocal for two, 1/a = b / (ab).
//              The exponent of 2 is cut at 60, which keeps the product finite (at 126 where
//              a value has its own reciprocal), and the factor z at -128, where the
//              exponent has long been cut: the result there is under 2^-53, however
//              negative z is.
//   gelu       z Phi(z) = max(z, 0) - u Phi(-u) with u = |z|, Phi the normal
//              distribution function, whose log2 Phi(-u) is smooth: a polynomial of
//              degree 7, a least-squares fit over 0 <= u <= 6 reweighted towards the
//              largest error, gives Phi(-u) to a relative 3.3e-6 (6.6e-6 evaluated in
//              fp32) with one exponential.  The pair form cuts u at 6: u Phi(-u) is below
//              6e-9 from there on, under half of fp16's least step, and nothing multiplies it.
//              The form for one value, which a gate may multiply by anything, goes on with
//              u Phi(-u) = phi(u) Q(1 / u^2) from 6 on, phi the normal density and Q a
//              least-squares fit of degree 3 (relative 1.1e-7; 8e-6 evaluated in fp32, where
//              the roundings of the exponent, up to 126, are most of it) down to 2^-126.
// The pair forms do the multiply-adds of two values in one instruction
// (f32x2, the same roundings).  4096 x 8192 x 256 with bias, where the epilogue is all
// the time: none 32 us, SILU 39, GELU 42, GELU_TANH 40.
// NaN stays NaN.
#pragma once

#include <cstdint>

namespace fp8q {

enum Activation : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger value, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Two fp32 values in one 64-bit register; element-wise operations, each value
// rounded to nearest.
typedef unsigned long long F32x2;
__device__ __forceinline__ F32x2 pack2(float a, float b) {
  F32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(F32x2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F32x2 mul2(F32x2 a, F32x2 b) {
  F32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F32x2 add2(F32x2 a, F32x2 b) {
  F32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F32x2 fma2(F32x2 a, F32x2 b, F32x2 c) {
  F32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F32x2 both(float a) { return pack2(a, a); }

constexpr float kLog2e = 1.44269504088896f;
// -2 u log2(e) = z (kTanh0 + kTanh1 z^2)
constexpr float kTanh0 = -1.59576912160573f * kLog2e;    // -2 sqrt(2/pi) log2(e)
constexpr float kTanh1 = -0.0713548162726009f * kLog2e;  // the same times 0.044715
constexpr float kGateCut = 60.0f;     // two values to a reciprocal
constexpr float kGateCutOne = 126.0f;
constexpr float kGateFloor = -128.0f;
constexpr float kGeluCut = 6.0f;
// log2 Phi(-u) = kGelu0 + u (kGelu1 + ..)
constexpr float kGelu0 = -0.999995294f, kGelu1 = -1.15125105f, kGelu2 = -0.458464391f, kGelu3 = -0.0539600711f,
                kGelu4 = 0.00850789188f, kGelu5 = -0.000930525087f, kGelu6 = 6.15983236e-05f, kGelu7 = -1.83481289e-06f;
// log2 phi(u) = kPhi0 + kPhi1 u^2,  Q(w) = kTail0 + w (kTail1 + ..)
constexpr float kPhi0 = -1.32574806f, kPhi1 = -0.5f * kLog2e;
constexpr float kTail0 = 0.999997139f, kTail1 = -0.999070108f, kTail2 = 2.89569616f, kTail3 = -9.96920872f;

// z / (1 + 2^e2)
__device__ __forceinline__ F32x2 gate2(F32x2 z, F32x2 e2) {
  float a, b;
  unpack2(z, a, b);
  z = pack2(max_nan(a, kGateFloor), max_nan(b, kGateFloor));
  unpack2(e2, a, b);
  unpack2(add2(pack2(ex2_approx(fminf(a, kGateCut)), ex2_approx(fminf(b, kGateCut))), both(1.0f)), a, b);
  return mul2(z, mul2(both(rcp_approx(__fmul_rn(a, b))), pack2(b, a)));
}

// ACT on two values.
template <int ACT>
__device__ __forceinline__ F32x2 activate2(F32x2 z) {
  if (ACT == kActNone) return z;
  if (ACT == kActSilu) return gate2(z, mul2(z, both(-kLog2e)));
  if (ACT == kActGeluTanh) return gate2(z, mul2(z, fma2(mul2(z, z), both(kTanh1), both(kTanh0))));
  float z0, z1;
  unpack2(z, z0, z1);
  const float r0 = max_nan(z0, 0.0f), r1 = max_nan(z1, 0.0f);
  if (ACT == kActRelu) return pack2(r0, r1);
  const F32x2 u = pack2(fminf(fabsf(z0), kGeluCut), fminf(fabsf(z1), kGeluCut));
  F32x2 q = fma2(u, both(kGelu7), both(kGelu6));
  q = fma2(q, u, both(kGelu5));
  q = fma2(q, u, both(kGelu4));
  q = fma2(q, u, both(kGelu3));
  q = fma2(q, u, both(kGelu2));
  q = fma2(q, u, both(kGelu1));
  q = fma2(q, u, both(kGelu0));
  float a, b;
  unpack2(q, a, b);
  q = pack2(ex2_approx(a), ex2_approx(b));               // Phi(-u)
  return fma2(mul2(u, both(-1.0f)), q, pack2(r0, r1));
}

// The activation `act` on one value (uniform over the grid: one branch), by the
// same formulas.
__device__ __forceinline__ float activate(float z, int act) {
  if (act == kActNone) return z;
  const float r = max_nan(z, 0.0f);
  if (act == kActRelu) return r;
  if (act == kActGelu) {
    const float u = fabsf(z);
    float f = u, q;   // u Phi(-u) = f 2^q
    if (u < kGeluCut) {
      q = fmaf(u, kGelu7, kGelu6);
      q = fmaf(q, u, kGelu5);
      q = fmaf(q, u, kGelu4);
      q = fmaf(q, u, kGelu3);
      q = fmaf(q, u, kGelu2);
      q = fmaf(q, u, kGelu1);
      q = fmaf(q, u, kGelu0);
    } else {
      const float t = __fmul_rn(u, u), w = rcp_approx(t);
      f = fmaf(fmaf(fmaf(kTail3, w, kTail2), w, kTail1), w, kTail0);
      q = fmaf(t, kPhi1, kPhi0);
    }
    return fmaf(-f, ex2_approx(q), r);
  }
  const float e = act == kActSilu ? __fmul_rn(z, -kLog2e) : __fmul_rn(z, fmaf(__fmul_rn(z, z), kTanh1, kTanh0));
  return __fmul_rn(max_nan(z, kGateFloor), rcp_approx(__fadd_rn(ex2_approx(fminf(e, kGateCutOne)), 1.0f)));
}

}  // namespace fp8q
