// Linear layers of up to 16 inputs (a few descriptors to features, the outer
// products of a readout's gradient): a tile of the tensor core's kernels would be
// mostly zeros, and the results are what takes the time.  A lane keeps the weights of
// one column, or of four where rows allow 16-byte pieces, in registers and goes down
// the rows, four of them in flight; a CTA stages 128 rows of x at a time in shared
// memory as fp32 (read back as broadcasts).  fp32 multiply-add, any stride.
//   fp32 SiLU, against the kernels for any K: 117,206 x 2 -> 21 8 us (25; its bytes
//   take 1.7), 131,072 x 4 -> 512 56 us (127; bytes 41), x 16 -> 512 103 us (128): the
//   instructions bound it there.
#include <algorithm>

#include "linear_epi.cuh"

namespace e2f {
namespace lin {
namespace thin {

constexpr int NT = 256, NW = NT / 32, ROWS = 128;

template <int CPL> __device__ __forceinline__ void load_extra4(float (&y)[CPL], const Epi &e, size_t i) {
  if constexpr (CPL == 1) {
    y[0] = load_as(e.extra, e.etype, i);
  } else if (e.etype == E2F_F32) {
    const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(e.extra) + i);
    y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(e.extra) + i);
    y[0] = __uint_as_float(v.x << 16); y[1] = __uint_as_float(v.x & 0xffff0000u);
    y[2] = __uint_as_float(v.y << 16); y[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
template <int CPL> __device__ __forceinline__ void store_out(const Epi &e, size_t i, const float (&v)[CPL]) {
  if constexpr (CPL == 1) {
    store_as(e.out, e.otype, i, v[0]);
  } else if (e.otype == E2F_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(e.out) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(e.out) + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// ... of dz in two bf16 terms, where it has them.
template <int CPL> __device__ __forceinline__ void store_dz(const Epi &e, size_t i, const float (&v)[CPL]) {
  if (!e.out2) {
    store_out<CPL>(e, i, v);
    return;
  }
  __nv_bfloat16 *h = static_cast<__nv_bfloat16 *>(e.out) + i, *l = static_cast<__nv_bfloat16 *>(e.out2) + i;
  if constexpr (CPL == 1) {
    two_terms(v[0], *h, *l);
  } else {
    uint2 a, b;
    two_terms({v[0], v[1]}, a.x, b.x);
    two_terms({v[2], v[3]}, a.y, b.y);
    *reinterpret_cast<uint2 *>(h) = a;
    *reinterpret_cast<uint2 *>(l) = b;
  }
}

// KP: inputs, rounded up; CPL: columns a lane; EXTRA: a residual or dL/dout is read.
template <typename T, int KP, int CPL, bool EXTRA>
__global__ void __launch_bounds__(NT) thin_kernel(const __grid_constant__ Gemm g) {
  constexpr int U = 4;
  __shared__ __align__(16) float sx[ROWS][KP];
  __shared__ __align__(16) float sw[KP][32 * CPL];
  __shared__ float red[NW][32 * CPL];
  after_previous();
  const Epi &e = g.e;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const T *B = static_cast<const T *>(g.B);
  const int n0 = blockIdx.y * (32 * CPL), n = n0 + lane * CPL;
  const bool in = n < g.N;   // (CPL divides N)
  for (int j = t; j < 32 * CPL * KP; j += NT) {
    const int c = j / KP, k = j % KP;
    sw[k][c] = n0 + c < g.N && k < g.K ? to_f(B[(size_t)((n0 + c) * g.ldb) + k]) : 0.f;
  }
  __syncthreads();
  float w[CPL][KP], bias[CPL], csum[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
#pragma unroll
    for (int k = 0; k < KP; ++k) w[c][k] = sw[k][lane * CPL + c];
    bias[c] = in && e.bias ? __ldg(e.bias + n + c) : 0.f;
    csum[c] = 0.f;
  }
  const int tiles = (g.M + ROWS - 1) / ROWS;
  for (int i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int m0 = i * ROWS, rows = min(ROWS, g.M - m0);
    const T *A = static_cast<const T *>(g.A) + (size_t)(m0 * g.lda);
    __syncthreads();
    for (int j = t; j < ROWS * KP; j += NT) {
      const int r = j / KP, k = j % KP;
      sx[r][k] = r < rows && k < g.K ? to_f(A[(size_t)(r * g.lda) + k]) : 0.f;
    }
    __syncthreads();
    for (int r0 = warp; r0 < rows && in; r0 += NW * U) {
      float y[U][CPL];
      if (EXTRA) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r0 + u * NW < rows) load_extra4<CPL>(y[u], e, (size_t)((long long)(m0 + r0 + u * NW) * e.lde) + n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * NW;
        if (r >= rows) break;
        float v[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) v[c] = 0.f;
#pragma unroll
        for (int k = 0; k < KP; k += 4) {
          const float4 x4 = *reinterpret_cast<const float4 *>(&sx[r][k]);
          const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (CPL == 1) {
              v[0] = fmaf(x[i], w[0][k + i], v[0]);
            } else {
#pragma unroll
              for (int c = 0; c < CPL; c += 2) {
                const f2 p = fma2(both(x[i]), {w[c][k + i], w[c + 1][k + i]}, {v[c], v[c + 1]});
                v[c] = p.x;
                v[c + 1] = p.y;
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) v[c] += bias[c];
        if (e.mode == MODE_DZ) {
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            v[c] = __fmul_rn(act_bwd(e.act, v[c]), EXTRA ? y[u][c] : 0.f);
            csum[c] += v[c];
          }
        } else {
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            v[c] = act_fwd(e.act, v[c]);
            if (EXTRA) v[c] += y[u][c];
          }
        }
        const size_t at = (size_t)((long long)(m0 + r) * e.ldo) + n;
        if (EXTRA && e.mode == MODE_DZ) {
          if (e.out) store_dz<CPL>(e, at, v);
        } else {
          store_out<CPL>(e, at, v);
        }
      }
    }
  }
  if (EXTRA && e.mode == MODE_DZ && e.colpart) {   // one partial row a CTA
#pragma unroll
    for (int c = 0; c < CPL; ++c) red[warp][lane * CPL + c] = csum[c];
    __syncthreads();
    if (t < 32 * CPL && n0 + t < g.N) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NW; ++j) s += red[j][t];
      e.colpart[(size_t)blockIdx.x * g.N + n0 + t] = s;
    }
  }
}

template <typename T, int KP, int CPL> static e2f_status launch(const Gemm &g, cudaStream_t s, int *rows_out) {
  // a block of columns and every gx-th block of rows to a CTA: the weights, whose
  // rows are apart, are read once
  const int cb = (g.N + 32 * CPL - 1) / (32 * CPL), gx = std::min((g.M + ROWS - 1) / ROWS, std::max(1, 1184 / cb));
  const dim3 grid((unsigned)gx, (unsigned)cb);
  if (rows_out) *rows_out = gx;
  if (g.e.extra) E2F_LIN_LAUNCH(g, (thin_kernel<T, KP, CPL, true>), grid, NT, 0, s, g);
  else E2F_LIN_LAUNCH(g, (thin_kernel<T, KP, CPL, false>), grid, NT, 0, s, g);
  return E2F_OK;
}
template <typename T, int KP> static e2f_status pick(const Gemm &g, cudaStream_t s, int *rows_out) {
  const Epi &e = g.e;
  const bool vec = g.N % 4 == 0 && g.N >= 96 && (!e.out || rows16(e.out, e.ldo, e.otype)) &&
                   (!e.extra || rows16(e.extra, e.lde, e.etype));
  return vec ? launch<T, KP, 4>(g, s, rows_out) : launch<T, KP, 1>(g, s, rows_out);
}

}  // namespace thin

// x W^T of up to 16 inputs, both K-major.
template <typename T> e2f_status gemm_thin(const Gemm &g, cudaStream_t s, int *rows_out) {
  if (g.K <= 4) return thin::pick<T, 4>(g, s, rows_out);
  if (g.K <= 8) return thin::pick<T, 8>(g, s, rows_out);
  return thin::pick<T, 16>(g, s, rows_out);
}
template e2f_status gemm_thin<float>(const Gemm &, cudaStream_t, int *);
template e2f_status gemm_thin<__nv_bfloat16>(const Gemm &, cudaStream_t, int *);

}  // namespace lin
}  // namespace e2f
