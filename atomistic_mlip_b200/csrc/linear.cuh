// Shared parts of the linear layer's kernels: the product's description, the
// epilogue applied to its accumulators, activations.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

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
  long long ldo;
  int otype;
  float *colpart;   // MODE_DZ: column sums of out per row block, fp32 [row blocks][N], or absent
};

// D[m][n] = sum_k A(m, k) B(n, k).  K-major: A(m, k) = A[m lda + k]; M-major:
// A(m, k) = A[k lda + m]; the same for B.
struct Gemm {
  const void *A, *B;
  long long lda, ldb;
  int M, N, K;
  int kper;          // contraction blocks (of BK) per split
  float *part;       // MODE_PART
  Epi e;
};

// sigma(z) = 1 / (1 + e^-z) by the special-function unit (2 instructions of it):
// good to about 2^-21, and e^-z = inf gives 0
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
__device__ __forceinline__ float silu_grad(float z) {
  const float s = sigmoid(z);
  return s * (1.f + z * (1.f - s));
}
// Phi(z), the normal distribution function, from Abramowitz and Stegun's
// rational approximation 7.1.26 of erfc(x) = t (a1 + t (a2 + ...)) e^(-x^2),
// t = 1 / (1 + p x) for x >= 0 (absolute error 1.5e-7, so 0.75e-7 in Phi), with
// x = |z| / sqrt 2; *e gets e^(-z^2 / 2), which the gradient needs as well.
// A third of erfcf's instructions, which bounded the epilogue (8,192 x 4,096 ->
// 4,096: 202 us with erfcf, 178 us without any activation).
__device__ __forceinline__ float normal_cdf(float z, float *e) {
  const float x = 0.70710678f * fabsf(z);
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  const float ex = __expf(-x * x);
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q *= 0.5f * t * ex;   // Phi(-|z|)
  *e = ex;
  return z < 0.f ? q : 1.f - q;
}
__device__ __forceinline__ float gelu(float z) {
  float e;
  return z * normal_cdf(z, &e);
}
__device__ __forceinline__ float gelu_grad(float z) {
  float e;
  const float p = normal_cdf(z, &e);
  return fmaf(0.39894228f * z, e, p);
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
__device__ __forceinline__ float epi_elem(const Epi &e, long long m, int n, float v, float bias) {
  v += bias;
  if (e.mode == MODE_OUT) {
    v = act_fwd(e.act, v);
    if (e.extra) v += load_as(e.extra, e.etype, (size_t)(m * e.lde) + n);
    store_as(e.out, e.otype, (size_t)(m * e.ldo) + n, v);
    return 0.f;
  }
  v = act_bwd(e.act, v) * load_as(e.extra, e.etype, (size_t)(m * e.lde) + n);
  if (e.out) store_as(e.out, e.otype, (size_t)(m * e.ldo) + n, v);
  return v;
}

}  // namespace lin
}  // namespace e2f
