// Linear layers with at most eight rows (a serving step) or at most eight
// outputs (the last layer of a readout): no tile to fill, the larger operand is
// streamed once and bounds the time.
//
// The streamed rows are W's (few x rows) or x's (few outputs).  LPR lanes share
// one of them, 32 / LPR rows a warp; every lane holds R partial sums, one per
// row of the small operand, which waits in shared memory as fp32, KC columns at
// a time.  The sums are joined by shuffles in a fixed order.  fp32 and bf16
// multiply in fp32 here.
#include <algorithm>

#include "linear.cuh"

namespace e2f {
namespace lin {
namespace skinny {

constexpr int NT = 256, NW = NT / 32, KC = 1024;

struct Args {
  Gemm g;
  bool outs;       // the small operand is W (few outputs), not x
  int lpr_log2;    // lanes per streamed row
  int iters;       // row groups a CTA takes one after another
};

template <typename T, int VE> __device__ __forceinline__ void load_ve(const T *p, float (&v)[VE]) {
  if constexpr (VE == 1) {
    v[0] = to_f(*p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 t = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u4w(t, i) << 16);
      v[2 * i + 1] = __uint_as_float(u4w(t, i) & 0xffff0000u);
    }
  }
}

// VE: elements of a streamed row a load takes (16 bytes, or 1 at any alignment).
template <typename T, int R, int VE>
__global__ void __launch_bounds__(NT) skinny_kernel(const __grid_constant__ Args a) {
  __shared__ float sm[R][KC];
  __shared__ float red[NW][R];
  after_previous();
  const Gemm &g = a.g;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int LPR = 1 << a.lpr_log2, li = lane & (LPR - 1), RW = 32 >> a.lpr_log2;
  const T *S = static_cast<const T *>(a.outs ? g.A : g.B), *P = static_cast<const T *>(a.outs ? g.B : g.A);
  const long long lds = a.outs ? g.lda : g.ldb, ldp = a.outs ? g.ldb : g.lda;
  const int rows = a.outs ? g.M : g.N, r = a.outs ? g.N : g.M;
  const int nchunk = (g.K + KC - 1) / KC;
  float csum[R];
#pragma unroll
  for (int j = 0; j < R; ++j) csum[j] = 0.f;
  for (int it = 0; it < a.iters; ++it) {
    const long long row = ((long long)blockIdx.x * a.iters + it) * (NW * RW) + warp * RW + (lane >> a.lpr_log2);
    const bool live = row < rows;
    const T *srow = S + (live ? (size_t)(row * lds) : 0);
    float acc[R];
#pragma unroll
    for (int j = 0; j < R; ++j) acc[j] = 0.f;
    for (int c = 0; c < nchunk; ++c) {
      const int k0 = c * KC, kn = min(KC, g.K - k0);
      constexpr int U = VE == 1 ? 8 : 4;   // loads in flight
      const int step = LPR * VE;
      float v[U][VE];
      auto fetch = [&](int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int e = 0; e < VE; ++e) v[u][e] = 0.f;
          if (live && k + u * step < kn) load_ve<T, VE>(srow + k0 + k + u * step, v[u]);
        }
      };
      fetch(li * VE);   // under way while the small operand is staged
      if (nchunk > 1 || it == 0) {
        __syncthreads();
        for (int i = t; i < R * KC; i += NT) {
          const int j = i / KC, k = i - j * KC;
          if (k < kn) sm[j][k] = j < r ? to_f(P[(size_t)(j * ldp) + k0 + k]) : 0.f;
        }
        __syncthreads();
      }
      for (int k = li * VE; k < kn; k += U * step) {
        if (k != li * VE) fetch(k);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int ku = k + u * step;
          if (ku >= kn) break;
#pragma unroll
          for (int j = 0; j < R; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) acc[j] = fmaf(v[u][e], sm[j][ku + e], acc[j]);
        }
      }
    }
    for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
      for (int j = 0; j < R; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    float rsum = 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (j < r && live && (j & (LPR - 1)) == li) {
        const int n = a.outs ? j : (int)row;
        const float d = epi_elem(g.e, a.outs ? row : j, n, acc[j], g.e.bias ? __ldg(g.e.bias + n) : 0.f);
        csum[j] += d;
        rsum += d;
      }
    }
    if (g.e.mode == MODE_DZ && g.e.colpart && !a.outs) {   // a column's rows are the lanes of one streamed row
      for (int o = 1; o < LPR; o <<= 1) rsum += __shfl_xor_sync(0xffffffffu, rsum, o);
      if (live && li == 0) g.e.colpart[row] = rsum;
    }
  }
  if (g.e.mode == MODE_DZ && g.e.colpart && a.outs) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float s = warp_sum(csum[j]);
      if (lane == 0) red[warp][j] = s;
    }
    __syncthreads();
    if (t < r) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s += red[w][t];
      g.e.colpart[(size_t)blockIdx.x * r + t] = s;
    }
  }
}

template <typename T, int R> static e2f_status launch(Args a, cudaStream_t s, int *rows_out) {
  const Gemm &g = a.g;
  constexpr int W = 16 / (int)sizeof(T);
  const void *S = a.outs ? g.A : g.B;
  const long long lds = a.outs ? g.lda : g.ldb;
  const bool vec = g.K % W == 0 && ((reinterpret_cast<uintptr_t>(S) | (uintptr_t)(lds * sizeof(T))) & 15) == 0;
  const int nv = vec ? g.K / W : g.K;
  a.lpr_log2 = 0;
  while (a.lpr_log2 < 5 && (1 << a.lpr_log2) < nv) ++a.lpr_log2;
  const int rows = a.outs ? g.M : g.N, group = NW * (32 >> a.lpr_log2);
  // Many rows: several groups to a CTA, which stages the small operand once.
  a.iters = (int)std::min<long long>(16, std::max<long long>(1, (long long)rows / (group * 1184LL)));
  const long long grid = ((long long)rows + group * a.iters - 1) / (group * a.iters);
  if (rows_out) *rows_out = a.outs ? (int)grid : 1;
  if (vec) E2F_LIN_LAUNCH(g, (skinny_kernel<T, R, W>), (unsigned)grid, NT, 0, s, a);
  else E2F_LIN_LAUNCH(g, (skinny_kernel<T, R, 1>), (unsigned)grid, NT, 0, s, a);
  return E2F_OK;
}

}  // namespace skinny

// x W^T with M or N up to 8, both K-major.
template <typename T> e2f_status gemm_skinny(const Gemm &g, cudaStream_t s, int *rows_out) {
  skinny::Args a{};
  a.g = g;
  a.outs = g.M > 8 || (g.N <= 8 && g.M > g.N);
  const int r = a.outs ? g.N : g.M;
  if (r == 1) return skinny::launch<T, 1>(a, s, rows_out);
  if (r == 2) return skinny::launch<T, 2>(a, s, rows_out);
  if (r <= 4) return skinny::launch<T, 4>(a, s, rows_out);
  return skinny::launch<T, 8>(a, s, rows_out);
}
template e2f_status gemm_skinny<float>(const Gemm &, cudaStream_t, int *);
template e2f_status gemm_skinny<__nv_bfloat16>(const Gemm &, cudaStream_t, int *);

}  // namespace lin
}  // namespace e2f
