// Linear layers with one or two rows (a serving step) or outputs (the last layer
// of a readout): no tile to fill, the larger operand is streamed once and bounds
// the time.  (From three on the tiled kernels win: at eight rows of 4,096 x 4,096
// bf16 the reads of the small operand took 120 us here, 16 us there.)
//
// The streamed rows are W's (few x rows) or x's (few outputs).  LPR lanes share
// RPT of them, RPT * 32 / LPR rows a warp; every lane holds RPT x R partial sums,
// R rows of the small operand, which waits in shared memory as fp32, KC columns
// at a time (eight consecutive ones in two halves, so that the lanes' 16-byte
// reads do not meet in a bank).  Four rows a lane read each of its values once
// for all four and keep four loads in flight where a row is short; one row a lane
// where there would not be CTAs enough.  The sums are joined by shuffles in a
// fixed order.  fp32 and bf16 multiply in fp32 here.
// Measured: 1 x 1,024 -> 4,096 bf16 5.3 us, most of it the latency of one pass;
// 100,002 x 1,000 -> 2 fp32 92 us (4.4 TB/s).
#include <algorithm>

#include "linear.cuh"

namespace e2f {
namespace lin {
namespace skinny {

constexpr int NT = 256, NW = NT / 32, KC = 4096;

struct Args {
  Gemm g;
  bool outs;       // the small operand is W (few outputs), not x
  int lpr_log2;    // lanes per streamed row
  int iters;       // row groups a CTA takes one after another
};

// VE consecutive elements of a streamed row as loaded, and as floats.
template <typename T, int VE> struct Piece {
  T v;
  __device__ __forceinline__ void zero() { v = from_f<T>(0.f); }
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void to(float (&f)[1]) const { f[0] = to_f(v); }
};
template <> struct Piece<float, 4> {
  float4 v;
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *p) { v = __ldg(reinterpret_cast<const float4 *>(p)); }
  __device__ __forceinline__ void to(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <> struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u4w(v, i) << 16);
      f[2 * i + 1] = __uint_as_float(u4w(v, i) & 0xffff0000u);
    }
  }
};

// VE: elements of a streamed row a load takes (16 bytes, or 1 at any alignment).
template <typename T, int R, int VE, int RPT>
__global__ void __launch_bounds__(NT) skinny_kernel(const __grid_constant__ Args a) {
  __shared__ __align__(16) float sm[R][KC];
  __shared__ float red[NW][R];
  after_previous();
  const Gemm &g = a.g;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int LPR = 1 << a.lpr_log2, li = lane & (LPR - 1), RW = 32 >> a.lpr_log2;
  const T *S = static_cast<const T *>(a.outs ? g.A : g.B), *P = static_cast<const T *>(a.outs ? g.B : g.A);
  const long long lds = a.outs ? g.lda : g.ldb, ldp = a.outs ? g.ldb : g.lda;
  const int rows = a.outs ? g.M : g.N, r = a.outs ? g.N : g.M;
  const int nchunk = (g.K + KC - 1) / KC;
  constexpr int U = (VE == 1 ? 8 : 4) / (RPT == 1 ? 1 : 2);   // loads of a row in flight
  float csum[R];
#pragma unroll
  for (int j = 0; j < R; ++j) csum[j] = 0.f;
  for (int it = 0; it < a.iters; ++it) {
    const long long row0 = (((long long)blockIdx.x * a.iters + it) * (NW * RW) + warp * RW + (lane >> a.lpr_log2)) * RPT;
    float acc[RPT][R];
#pragma unroll
    for (int q = 0; q < RPT; ++q)
#pragma unroll
      for (int j = 0; j < R; ++j) acc[q][j] = 0.f;
    for (int c = 0; c < nchunk; ++c) {
      const int k0 = c * KC, kn = min(KC, g.K - k0);
      const int step = LPR * VE;
      Piece<T, VE> v[RPT][U];
      auto fetch = [&](int k) {
#pragma unroll
        for (int q = 0; q < RPT; ++q)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            v[q][u].zero();
            if (row0 + q < rows && k + u * step < kn) v[q][u].load(S + (size_t)((row0 + q) * lds) + k0 + k + u * step);
          }
      };
      fetch(li * VE);   // under way while the small operand is staged
      if (nchunk > 1 || it == 0) {
        __syncthreads();
        for (int i = t; i < R * kn; i += NT) {
          const int j = R == 1 || i < kn ? 0 : 1, k = i - j * kn;
          if (k < kn) sm[j][VE == 8 ? (k >> 3) * 4 + (k & 3) + ((k >> 2) & 1) * (KC / 2) : k] =
              j < r ? to_f(P[(size_t)(j * ldp) + k0 + k]) : 0.f;
        }
        __syncthreads();
      }
      for (int k = li * VE; k < kn; k += U * step) {
        if (k != li * VE) fetch(k);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int ku = k + u * step;
          if (ku >= kn) break;
          float f[RPT][VE];
#pragma unroll
          for (int q = 0; q < RPT; ++q) v[q][u].to(f[q]);
#pragma unroll
          for (int j = 0; j < R; ++j) {
            float p[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) p[e] = VE == 8 ? sm[j][(ku >> 1) + (e & 3) + (e >> 2) * (KC / 2)] : sm[j][ku + e];
#pragma unroll
            for (int q = 0; q < RPT; ++q)
#pragma unroll
              for (int e = 0; e < VE; ++e) acc[q][j] = fmaf(f[q][e], p[e], acc[q][j]);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < RPT; ++q) {
      const long long row = row0 + q;
      const bool live = row < rows;
      for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
        for (int j = 0; j < R; ++j) acc[q][j] += __shfl_xor_sync(0xffffffffu, acc[q][j], o);
      float rsum = 0.f;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (j < r && live && (j & (LPR - 1)) == li) {
          const int n = a.outs ? j : (int)row;
          const float d = epi_elem(g.e, a.outs ? row : j, n, acc[q][j], g.e.bias ? __ldg(g.e.bias + n) : 0.f);
          csum[j] += d;
          rsum += d;
        }
      }
      if (g.e.mode == MODE_DZ && g.e.colpart && !a.outs) {   // a column's rows are the lanes of one streamed row
        for (int o = 1; o < LPR; o <<= 1) rsum += __shfl_xor_sync(0xffffffffu, rsum, o);
        if (live && li == 0) g.e.colpart[row] = rsum;
      }
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

template <typename T, int R, int VE, int RPT> static e2f_status launch_rpt(Args a, cudaStream_t s, int *rows_out) {
  const Gemm &g = a.g;
  const int rows = a.outs ? g.M : g.N, group = NW * (32 >> a.lpr_log2) * RPT;
  // Many rows: several groups to a CTA, which stages the small operand once.
  a.iters = (int)std::min<long long>(16, std::max<long long>(1, (long long)rows / (group * 1184LL)));
  const long long grid = ((long long)rows + (long long)group * a.iters - 1) / ((long long)group * a.iters);
  if (rows_out) *rows_out = a.outs ? (int)grid : 1;
  E2F_LIN_LAUNCH(g, (skinny_kernel<T, R, VE, RPT>), (unsigned)grid, NT, 0, s, a);
  return E2F_OK;
}

template <typename T, int R> static e2f_status launch(Args a, cudaStream_t s, int *rows_out) {
  const Gemm &g = a.g;
  constexpr int W = 16 / (int)sizeof(T);
  const void *S = a.outs ? g.A : g.B;
  const long long lds = a.outs ? g.lda : g.ldb;
  const bool vec = g.K % W == 0 && ((reinterpret_cast<uintptr_t>(S) | (uintptr_t)(lds * sizeof(T))) & 15) == 0;
  const int nv = vec ? g.K / W : g.K;
  // two to four loads of a row to a lane: fewer shuffles and epilogues a warp than
  // with one
  a.lpr_log2 = 0;
  while (a.lpr_log2 < 5 && (4 << a.lpr_log2) < nv) ++a.lpr_log2;
  const int rows = a.outs ? g.M : g.N;
  const bool four = rows >= 148 * NW * (32 >> a.lpr_log2) * 4;   // a CTA on every SM all the same
  if (vec) return four ? launch_rpt<T, R, W, 4>(a, s, rows_out) : launch_rpt<T, R, W, 1>(a, s, rows_out);
  return four ? launch_rpt<T, R, 1, 4>(a, s, rows_out) : launch_rpt<T, R, 1, 1>(a, s, rows_out);
}

}  // namespace skinny

// x W^T with M or N up to 2, both K-major.
template <typename T> e2f_status gemm_skinny(const Gemm &g, cudaStream_t s, int *rows_out) {
  skinny::Args a{};
  a.g = g;
  a.outs = g.M > 2 || (g.N <= 2 && g.M > g.N);
  return (a.outs ? g.N : g.M) == 1 ? skinny::launch<T, 1>(a, s, rows_out) : skinny::launch<T, 2>(a, s, rows_out);
}
template e2f_status gemm_skinny<float>(const Gemm &, cudaStream_t, int *);
template e2f_status gemm_skinny<__nv_bfloat16>(const Gemm &, cudaStream_t, int *);

}  // namespace lin
}  // namespace e2f
