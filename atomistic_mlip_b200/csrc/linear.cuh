// Shared parts of the linear layer's kernels: the product's description, the
// epilogue applied to its accumulators, activations.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

// Launch by g.after: behind another kernel of the call, or in plain stream order.
#define E2F_LIN_LAUNCH(g, kernel, grid, block, smem, stream, ...)              \
  do {                                                                         \
    if ((g).after) E2F_LAUNCH_AFTER(kernel, grid, block, smem, stream, __VA_ARGS__); \
    else E2F_LAUNCH(kernel, grid, block, smem, stream, __VA_ARGS__);           \
  } while (0)

namespace e2f {
namespace lin {

// What becomes of an accumulator v of row m, column n.
constexpr int MODE_OUT = 0;    // out = act(v + bias) + extra        (extra: the residual, may be absent)
constexpr int MODE_DZ = 1;     // out = act'(v + bias) * extra       (extra: dL/dout; out may be absent)
constexpr int MODE_PART = 2;   // partial sum of a split contraction, fp32 [split][M][N]

struct Epi {
  int mode, act;
  const float *bias;
  const void *extra;
  long long lde;
  int etype;
  void *out;
  void *out2;       // MODE_DZ, bf16: what out leaves of the value, in bf16 and out's layout, or absent
  long long ldo;
  int otype;
  float *colpart;   // MODE_DZ: column sums of out per row block, fp32 [row blocks][N], or absent
};

// D[m][n] = sum_k A(m, k) B(n, k).  K-major: A(m, k) = A[m lda + k]; M-major:
// A(m, k) = A[k lda + m]; the same for B.
struct Gemm {
  const void *A, *B;
  const void *A2;    // bf16: a second term of A in the same layout (A + A2 is meant), or absent
  long long lda, ldb;
  int M, N, K;
  int kper;          // contraction blocks (of BK) per split
  float *part;       // MODE_PART
  bool after;        // launched behind another kernel of the call
  Epi e;
};

// 2^x and 1 / x by the special-function unit, one instruction each (2^-22 and
// one unit in the last place); denormal results are zero.
__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcpf(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float LOG2E = 1.44269504f;

// Each function stands here for one value and for two: the same operations with the
// same roundings, so that a pre-activation gives the same bits in every kernel
// (__fmul_rn: a product that the compiler does not fuse with an addition behind it).
// sigma(z) = 1 / (1 + e^-z); e^-z = inf gives 0
__device__ __forceinline__ float sigmoid(float z) { return rcpf(1.f + ex2f(-LOG2E * z)); }
__device__ __forceinline__ float silu(float z) { return __fmul_rn(z, sigmoid(z)); }
__device__ __forceinline__ float silu_grad(float z) {
  const float s = sigmoid(z);
  return fmaf(s * z, 1.f - s, s);
}
// Phi(z), the normal distribution function, from Abramowitz and Stegun's
// rational approximation 7.1.26 of erfc(x) = t (a1 + t (a2 + ...)) e^(-x^2),
// t = 1 / (1 + p x) for x >= 0 (absolute error 1.5e-7, so 0.75e-7 in Phi), with
// x = |z| / sqrt 2; *e gets e^(-z^2 / 2), which the gradient needs as well.
// A fraction of erfcf's instructions, which bounded the epilogue (8,192 x 4,096
// -> 4,096: 202 us with erfcf, 183 us so, 174 us without any activation).  In the
// lower tail it is off by 0.2 % at z = -5, 0.4 % at -6.
__device__ __forceinline__ float normal_cdf(float z, float *e) {
  const float t = rcpf(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.f));
  const float ex = ex2f(-0.5f * LOG2E * z * z);
  float q = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  q = fmaf(q, t, 0.5f * 1.421413741f);
  q = fmaf(q, t, 0.5f * -0.284496736f);
  q = fmaf(q, t, 0.5f * 0.254829592f);
  q = __fmul_rn(__fmul_rn(q, t), ex);   // Phi(-|z|)
  *e = ex;
  return z < 0.f ? q : 1.f - q;
}
__device__ __forceinline__ float gelu(float z) {
  float e;
  return __fmul_rn(z, normal_cdf(z, &e));
}
__device__ __forceinline__ float gelu_grad(float z) {
  float e;
  const float p = normal_cdf(z, &e);
  return fmaf(0.39894228f * z, e, p);
}
// ---- two at a time: one issue slot for two fp32 operations (the epilogues are
// bound by issue slots) -------------------------------------------------------------
struct f2 {
  float x, y;
};
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 s, p, q;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 s, p, q;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("{\n\t.reg .b64 p, q, t, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 t, {%6, %7};\n\t"
      "fma.rn.f32x2 s, p, q, t;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return {v, v}; }
// (One reciprocal for a pair, (1 / (d.x d.y)) d.y and the same by d.x, saves a
// special-function instruction in four but needs a guard against d.x d.y = inf:
// 100,002 x 128 -> 512 SiLU 47 us against 40.)
__device__ __forceinline__ f2 sigmoid(f2 z) {
  f2 e = mul2(z, both(-LOG2E));
  e = add2({ex2f(e.x), ex2f(e.y)}, both(1.f));
  return {rcpf(e.x), rcpf(e.y)};
}
__device__ __forceinline__ f2 silu(f2 z) { return mul2(z, sigmoid(z)); }
__device__ __forceinline__ f2 silu_grad(f2 z) {
  const f2 s = sigmoid(z);
  return fma2(mul2(s, z), fma2(s, both(-1.f), both(1.f)), s);
}
__device__ __forceinline__ f2 normal_cdf(f2 z, f2 *e) {
  f2 t = fma2({fabsf(z.x), fabsf(z.y)}, both(0.3275911f * 0.70710678f), both(1.f));
  t = {rcpf(t.x), rcpf(t.y)};
  f2 x = mul2(mul2(z, both(-0.5f * LOG2E)), z);
  x = {ex2f(x.x), ex2f(x.y)};
  f2 q = fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
  q = fma2(q, t, both(0.5f * 1.421413741f));
  q = fma2(q, t, both(0.5f * -0.284496736f));
  q = fma2(q, t, both(0.5f * 0.254829592f));
  q = mul2(mul2(q, t), mul2(x, both(-1.f)));   // -Phi(-|z|)
  *e = x;
  const f2 s = {copysignf(1.f, z.x), copysignf(1.f, z.y)};
  return fma2(q, s, fma2(s, both(0.5f), both(0.5f)));   // z < 0: 0 + Phi(-|z|), else 1 - Phi(-|z|)
}
__device__ __forceinline__ f2 gelu(f2 z) {
  f2 e;
  return mul2(z, normal_cdf(z, &e));
}
__device__ __forceinline__ f2 gelu_grad(f2 z) {
  f2 e;
  const f2 p = normal_cdf(z, &e);
  return fma2(mul2(z, both(0.39894228f)), e, p);
}

// Two bf16 terms of each of a pair, together 16 bits: h the nearest, l what it leaves
// (nothing where h is not finite).
__device__ __forceinline__ void two_terms(f2 v, uint32_t &h, uint32_t &l) {
  h = pack_bf16x2(v.x, v.y);
  const f2 r = fma2({__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)}, both(-1.f), v);
  l = pack_bf16x2(fabsf(r.x) < INFINITY ? r.x : 0.f, fabsf(r.y) < INFINITY ? r.y : 0.f);
}
// The same of one value that may meet infinities in a product (dz = dL/dout, without
// an activation whose derivative would be NaN beside them): h is cut, not rounded, so
// that l has its sign, and l is zero only where h is: infinity times either of them
// is the same infinity.
__device__ __forceinline__ void two_terms(float v, __nv_bfloat16 &h, __nv_bfloat16 &l) {
  h = __float2bfloat16_rz(v);
  const float w = __bfloat162float(h);
  l = __float2bfloat16_rn(copysignf(fmaxf(fabsf(v - w), fabsf(w) * 0x1p-30f), v));
}

__device__ __forceinline__ float act_fwd(int act, float z) {
  return act == E2F_ACT_SILU ? silu(z) : act == E2F_ACT_GELU ? gelu(z) : z;
}
__device__ __forceinline__ float act_bwd(int act, float z) {
  return act == E2F_ACT_SILU ? silu_grad(z) : act == E2F_ACT_GELU ? gelu_grad(z) : 1.f;
}

__device__ __forceinline__ float load_as(const void *p, int type, size_t i) {
  return type == E2F_F32 ? static_cast<const float *>(p)[i] : to_f(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_as(void *p, int type, size_t i, float v) {
  if (type == E2F_F32) static_cast<float *>(p)[i] = v;
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// One element through the epilogue; returns what MODE_DZ adds to its column's sum.
// (The product is rounded before it is added: fused with the addition where dz is
// not stored as well, it would give the sums other bits there.)
__device__ __forceinline__ float epi_elem(const Epi &e, long long m, int n, float v, float bias) {
  v += bias;
  if (e.mode == MODE_OUT) {
    v = act_fwd(e.act, v);
    if (e.extra) v += load_as(e.extra, e.etype, (size_t)(m * e.lde) + n);
    store_as(e.out, e.otype, (size_t)(m * e.ldo) + n, v);
    return 0.f;
  }
  v = __fmul_rn(act_bwd(e.act, v), load_as(e.extra, e.etype, (size_t)(m * e.lde) + n));
  if (e.out) {
    const size_t i = (size_t)(m * e.ldo) + n;
    if (e.out2) two_terms(v, static_cast<__nv_bfloat16 *>(e.out)[i], static_cast<__nv_bfloat16 *>(e.out2)[i]);
    else store_as(e.out, e.otype, i, v);
  }
  return v;
}

}  // namespace lin
}  // namespace e2f
