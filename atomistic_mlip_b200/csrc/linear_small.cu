// Small linear layers on the CUDA cores: a few thousand outputs leave the tensor
// core's kernels nothing but their latency (8 to 10 us with fp32 operands).  A CTA
// has a 32 x 32 piece (fp32 multiply-add, 32 contraction steps at a time, the next
// ones on their way); shared-memory reads bound it, at a third of the fp32 rate.
//   small_kernel        x W^T with its epilogue (forward, dz; 3,000 x 128 -> 64 7.8 us)
//   small_grads_kernel  dx = dz W, dW = dz^T x and the bias's column sums in one
//                       launch (300 x 72 x 96 fp32: 24 us a call against 36)
#include <algorithm>

#include "linear.cuh"

namespace e2f {
namespace lin {
namespace small {

constexpr int NT = 256, TS = 32, PITCH = TS + 2;

// The value that two terms stand for (see two_terms: beside an infinite one the second
// adds nothing).
__device__ __forceinline__ float terms_sum(float h, float l) { return fabsf(h) < INFINITY ? h + l : h; }

// Four elements of a 32 x 32 operand piece (row r of r0 .., contraction k of
// k0 ..) a thread; CONTIG: the contraction index is the contiguous one.
// P2: a second term of every element, or null.
template <typename T, bool CONTIG>
__device__ __forceinline__ void fetch(float (&v)[4], const T *P, const T *P2, long long ld, int r0, int rn, int k0, int kn) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int f = threadIdx.x & 31, s = (threadIdx.x >> 5) + 8 * j;
    const int r = r0 + (CONTIG ? s : f), k = k0 + (CONTIG ? f : s);
    const size_t i = CONTIG ? (size_t)(r * ld) + k : (size_t)(k * ld) + r;
    v[j] = r < rn && k < kn ? to_f(P[i]) : 0.f;
    if (P2 && r < rn && k < kn) v[j] = terms_sum(v[j], to_f(P2[i]));
  }
}
template <bool CONTIG> __device__ __forceinline__ void put(const float (&v)[4], float (*s)[PITCH]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int f = threadIdx.x & 31, q = (threadIdx.x >> 5) + 8 * j;
    s[CONTIG ? f : q][CONTIG ? q : f] = v[j];   // [contraction][row]
  }
}

// acc[i][j] = sum_k A(r, k) B(c, k) for r = r0 + 2 (t / 16) + i, c = c0 + 2 (t % 16) + j.
template <typename T, bool A_CONTIG, bool B_CONTIG>
__device__ __forceinline__ void product(float (&acc)[2][2], const T *A, const T *A2, long long lda, const T *B, long long ldb,
                                        int r0, int rn, int c0, int cn, int kn, float (*sa)[PITCH], float (*sb)[PITCH]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float va[4], vb[4];
  acc[0][0] = acc[0][1] = acc[1][0] = acc[1][1] = 0.f;
  fetch<T, A_CONTIG>(va, A, A2, lda, r0, rn, 0, kn);
  fetch<T, B_CONTIG>(vb, B, static_cast<const T *>(nullptr), ldb, c0, cn, 0, kn);
  for (int k0 = 0; k0 < kn; k0 += TS) {
    __syncthreads();
    put<A_CONTIG>(va, sa);
    put<B_CONTIG>(vb, sb);
    __syncthreads();
    if (k0 + TS < kn) {
      fetch<T, A_CONTIG>(va, A, A2, lda, r0, rn, k0 + TS, kn);
      fetch<T, B_CONTIG>(vb, B, static_cast<const T *>(nullptr), ldb, c0, cn, k0 + TS, kn);
    }
#pragma unroll
    for (int k = 0; k < TS; ++k) {
      const float2 a = *reinterpret_cast<const float2 *>(&sa[k][2 * ty]), b = *reinterpret_cast<const float2 *>(&sb[k][2 * tx]);
      acc[0][0] = fmaf(a.x, b.x, acc[0][0]);
      acc[0][1] = fmaf(a.x, b.y, acc[0][1]);
      acc[1][0] = fmaf(a.y, b.x, acc[1][0]);
      acc[1][1] = fmaf(a.y, b.y, acc[1][1]);
    }
  }
}
template <typename T, bool A_CONTIG>
__device__ __forceinline__ void piece(const T *A, const T *A2, long long lda, const T *B, long long ldb, T *out,
                                      long long ldo, int r0, int rn, int c0, int cn, int kn, float (*sa)[PITCH], float (*sb)[PITCH]) {
  float acc[2][2];
  product<T, A_CONTIG, false>(acc, A, A2, lda, B, ldb, r0, rn, c0, cn, kn, sa, sb);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = r0 + 2 * (threadIdx.x >> 4) + i, c = c0 + 2 * (threadIdx.x & 15) + j;
      if (r < rn && c < cn) out[(size_t)(r * ldo) + c] = from_f<T>(acc[i][j]);
    }
}

template <typename T> __global__ void __launch_bounds__(NT) small_kernel(const __grid_constant__ Gemm g) {
  __shared__ float sa[TS][PITCH], sb[TS][PITCH];
  after_previous();
  const int nt = (g.N + TS - 1) / TS, r0 = blockIdx.x / nt * TS, c0 = blockIdx.x % nt * TS;
  float acc[2][2];
  product<T, true, true>(acc, static_cast<const T *>(g.A), nullptr, g.lda, static_cast<const T *>(g.B), g.ldb, r0, g.M, c0,
                         g.N, g.K, sa, sb);
  // lane = column through shared memory: rows out in contiguous pieces
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) sa[2 * (threadIdx.x >> 4) + i][2 * (threadIdx.x & 15) + j] = acc[i][j];
  __syncthreads();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = c0 + lane;
  float csum = 0.f;
  if (n < g.N) {
    const float bias = g.e.bias ? g.e.bias[n] : 0.f;
#pragma unroll
    for (int q = 0; q < TS / 8; ++q) {
      const int r = w + 8 * q;
      if (r0 + r < g.M) csum += epi_elem(g.e, r0 + r, n, sa[r][lane], bias);
    }
  }
  if (g.e.mode == MODE_DZ && g.e.colpart) {   // one partial row per 32 rows
    sb[w][lane] = csum;
    __syncthreads();
    if (w == 0 && n < g.N) {
#pragma unroll
      for (int j = 1; j < NT / 32; ++j) csum += sb[j][lane];
      g.e.colpart[(size_t)(r0 / TS) * g.N + n] = csum;
    }
  }
}

struct Args {
  const void *dz, *dz2, *x, *W;   // dz2: dz's second term, or null
  long long ldz, ldx, ldw;
  void *gx, *gW;
  long long ldgx, ldgw;
  int M, N, K;
  int nx, nw;          // CTAs of dx, of dW; the rest sum columns
  const void *cp;      // rows whose column sums are the bias's gradient
  int ctype, crows;
  long long cld;
  float *gb;
};

template <typename T> __global__ void __launch_bounds__(NT) small_grads_kernel(const __grid_constant__ Args a) {
  __shared__ float sa[TS][PITCH], sb[TS][PITCH];
  after_previous();
  const T *dz = static_cast<const T *>(a.dz), *dz2 = static_cast<const T *>(a.dz2);
  const T *x = static_cast<const T *>(a.x), *W = static_cast<const T *>(a.W);
  const int kt = (a.K + TS - 1) / TS;
  int b = blockIdx.x;
  if (b < a.nx) {
    piece<T, true>(dz, dz2, a.ldz, W, a.ldw, static_cast<T *>(a.gx), a.ldgx, b / kt * TS, a.M, b % kt * TS, a.K, a.N, sa, sb);
    return;
  }
  b -= a.nx;
  if (b < a.nw) {
    piece<T, false>(dz, dz2, a.ldz, x, a.ldx, static_cast<T *>(a.gW), a.ldgw, b / kt * TS, a.N, b % kt * TS, a.K, a.M, sa, sb);
    return;
  }
  b -= a.nw;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = b * 32 + lane;
  float s = 0.f;
  if (n < a.N)
#pragma unroll 8
    for (int i = w; i < a.crows; i += NT / 32) s += load_as(a.cp, a.ctype, (size_t)(i * a.cld) + n);
  sa[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < a.N) {
#pragma unroll
    for (int j = 1; j < NT / 32; ++j) s += sa[j][lane];
    a.gb[n] = s;
  }
}

}  // namespace small

// Pieces of the output, contraction steps and their product (what a CTA slot works
// through) up to limits.
static bool fits(int rows, int cols, int k, int kmax, long long pieces, long long work) {
  const long long p = (long long)((rows + 31) / 32) * ((cols + 31) / 32);
  return k <= kmax && p <= pieces && p * k <= work;
}
// Against the kernels with operands through registers (kernel times, fp32, SiLU):
// 64 pieces of 64 steps 4.7 and 8.0 us, 256 of 128 8 and 9.6, 128 of 256 9.8 and
// 12; behind the limits 512 of 128 12.5 and 9.7, 1,024 of 16 and a residual 12.5 and
// 9.6, 128 of 512 16 and 17, with a residual 19 and 18.  Against those fed by TMA
// (tma): 128 pieces of 16 steps 4.3 and 5.5 us, of 64 5.6 and 5.5, with a residual
// or dL/dout on vector rows (extra) of 16 6.5 and 5.7.
bool small_fit(int M, int N, int K, int dtype, bool tma, bool extra) {
  if (tma) return !extra && fits(M, N, K, 32, 256, 32768);
  return fits(M, N, K, dtype == E2F_F32 ? 256 : 128, 512, 32768);
}
// One launch for three: up to larger products (256 x 64 -> 128 fp32 with its dz 14
// and 35 us).
bool small_grads_fit(int M, int N, int K, int dtype) {
  const int kmax = dtype == E2F_F32 ? 512 : 128;
  return fits(M, K, N, kmax, 512, 65536) && fits(N, K, M, kmax, 512, 65536);
}

template <typename T> e2f_status gemm_small(const Gemm &g, cudaStream_t s) {
  const int grid = (g.M + 31) / 32 * ((g.N + 31) / 32);
  E2F_LIN_LAUNCH(g, small::small_kernel<T>, grid, small::NT, 0, s, g);
  return E2F_OK;
}
template e2f_status gemm_small<float>(const Gemm &, cudaStream_t);
template e2f_status gemm_small<__nv_bfloat16>(const Gemm &, cudaStream_t);

template <typename T>
e2f_status small_grads(const e2f_linear &p, const void *dz, const void *dz2, long long ldz, void *gx, long long ldgx, void *gW,
                       long long ldgw, const void *cp, int ctype, long long cld, int crows, float *gb, bool after, cudaStream_t s) {
  small::Args a{};
  a.dz = dz; a.dz2 = dz2; a.ldz = ldz; a.x = p.x; a.ldx = p.ldx; a.W = p.W; a.ldw = p.ldw;
  a.gx = gx; a.ldgx = ldgx; a.gW = gW; a.ldgw = ldgw;
  a.M = (int)p.M; a.N = p.N; a.K = p.K;
  const int kt = (p.K + 31) / 32;
  a.nx = gx ? (a.M + 31) / 32 * kt : 0;
  a.nw = gW ? (a.N + 31) / 32 * kt : 0;
  a.cp = cp; a.ctype = ctype; a.cld = cld; a.crows = crows; a.gb = gb;
  const int grid = a.nx + a.nw + (gb ? (a.N + 31) / 32 : 0);
  if (grid == 0) return E2F_OK;
  if (after) E2F_LAUNCH_AFTER(small::small_grads_kernel<T>, grid, small::NT, 0, s, a);
  else E2F_LAUNCH(small::small_grads_kernel<T>, grid, small::NT, 0, s, a);
  return E2F_OK;
}
template e2f_status small_grads<float>(const e2f_linear &, const void *, const void *, long long, void *, long long, void *,
                                       long long, const void *, int, long long, int, float *, bool, cudaStream_t);
template e2f_status small_grads<__nv_bfloat16>(const e2f_linear &, const void *, const void *, long long, void *, long long,
                                               void *, long long, const void *, int, long long, int, float *, bool,
                                               cudaStream_t);

}  // namespace lin
}  // namespace e2f
