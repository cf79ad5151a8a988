// Activations of the FFN epilogues (dense linear with an epilogue, MoE layer),
// in fp32 on values that are rounded to fp16 right after.
//
// Accuracy: the target is an error far under half an fp16 step (2^-11
// relative), at a cost that hides behind the tensor-core mainloop.  Each of the
// three smooth ones is two special-function operations (ex2.approx and
// rcp.approx, relative error about 2^-22 each) and a few multiply-adds:
//   silu       z / (1 + e^-z)
//   gelu_tanh  0.5 z (1 + tanh u) = z / (1 + e^-2u),  u = sqrt(2/pi) (z + 0.044715 z^3)
//   gelu       z Phi(z) = max(z, 0) - |z| Phi(-|z|), Phi the normal distribution
//              function: with u = |z| and t = 1 / (1 + 0.3 u),
//              Phi(-u) = e^(-u^2/2) t P(t).  P, of degree 5, is a least-squares fit
//              (reweighted towards the largest relative error) of
//              erfcx(u / sqrt(2)) / (2 t) over 0 <= u <= 9: relative error 2.1e-6, which
//              the factored exponential carries to the far negative tail (3.6e-6
//              relative in fp32 for |z| < 6, past which fp16 has no value left).
// The pair forms do the multiply-adds of two values in one instruction
// (f32x2, the same roundings): the large GEMM's epilogue has 32768 values a tile and
// SM, whose special functions take 4100 cycles and whose mainloop 8900 at K = 2048.
// NaN stays NaN; relu(-0) = -0.
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
constexpr float kGeluC = 0.3f;
constexpr float kGeluP0 = 0.120327727f, kGeluP1 = 0.111210456f, kGeluP2 = 0.153751159f, kGeluP3 = -0.0340378628f,
                kGeluP4 = 0.230586332f, kGeluP5 = -0.0818373346f;

// z times sigmoid, e2 = the exponent of 2 that is e^-x of the sigmoid's argument
__device__ __forceinline__ F32x2 gate2(F32x2 z, F32x2 e2) {
  float a, b;
  unpack2(e2, a, b);
  const F32x2 d = add2(pack2(ex2_approx(a), ex2_approx(b)), both(1.0f));
  unpack2(d, a, b);
  return mul2(z, pack2(rcp_approx(a), rcp_approx(b)));
}

// ACT on two values.
template <int ACT>
__device__ __forceinline__ F32x2 activate2(F32x2 z) {
  if (ACT == kActNone) return z;
  if (ACT == kActSilu) return gate2(z, mul2(z, both(-kLog2e)));
  if (ACT == kActGeluTanh) return gate2(z, mul2(z, fma2(mul2(z, z), both(kTanh1), both(kTanh0))));
  float z0, z1;
  unpack2(z, z0, z1);
  const float r0 = z0 < 0.0f ? 0.0f : z0, r1 = z1 < 0.0f ? 0.0f : z1;   // (NaN passes)
  if (ACT == kActRelu) return pack2(r0, r1);
  const F32x2 u = pack2(fabsf(z0), fabsf(z1));
  float a, b;
  unpack2(fma2(u, both(kGeluC), both(1.0f)), a, b);
  const F32x2 t = pack2(rcp_approx(a), rcp_approx(b));
  F32x2 q = fma2(t, both(kGeluP5), both(kGeluP4));
  q = fma2(q, t, both(kGeluP3));
  q = fma2(q, t, both(kGeluP2));
  q = fma2(q, t, both(kGeluP1));
  q = fma2(q, t, both(kGeluP0));
  const F32x2 minus_u = pack2(-fabsf(z0), -fabsf(z1));
  unpack2(mul2(mul2(u, both(0.5f * kLog2e)), minus_u), a, b);
  q = mul2(mul2(q, t), pack2(ex2_approx(a), ex2_approx(b)));   // Phi(-|z|)
  return fma2(minus_u, q, pack2(r0, r1));
}

// The activation `act` on one value (uniform over the grid: one branch); the
// same operations as a pair's.
__device__ __forceinline__ float activate(float z, int act) {
  if (act == kActNone) return z;
  const float r = z < 0.0f ? 0.0f : z;   // (NaN passes)
  if (act == kActRelu) return r;
  if (act == kActGelu) {
    const float u = fabsf(z), t = rcp_approx(fmaf(u, kGeluC, 1.0f));
    float q = fmaf(t, kGeluP5, kGeluP4);
    q = fmaf(q, t, kGeluP3);
    q = fmaf(q, t, kGeluP2);
    q = fmaf(q, t, kGeluP1);
    q = fmaf(q, t, kGeluP0);
    q = __fmul_rn(__fmul_rn(q, t), ex2_approx(__fmul_rn(__fmul_rn(u, 0.5f * kLog2e), -u)));
    return fmaf(-u, q, r);
  }
  const float e = act == kActSilu ? __fmul_rn(z, -kLog2e) : __fmul_rn(z, fmaf(__fmul_rn(z, z), kTanh1, kTanh0));
  return __fmul_rn(z, rcp_approx(__fadd_rn(ex2_approx(e), 1.0f)));
}

}  // namespace fp8q
