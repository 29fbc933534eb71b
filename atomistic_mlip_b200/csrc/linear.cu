// Linear layers with bias, activation and residual in the epilogue, and their
// gradient:
//
//   forward    y  = act(x W^T + b) + r
//   backward   z  = x W^T + b (formed again: nothing but y leaves the forward),
//              dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
//
// Products run on the tensor cores (linear_tma.cu, linear_reg.cu), but for those
// with one or two rows or outputs (linear_skinny.cu), up to 16 inputs
// (linear_thin.cu) or too few tiles to fill them (linear_small.cu).  bf16 operands are used as they are, fp32
// accumulation.  fp32 operands are split into three bf16 terms each,
// x = h + m + l (8 + 8 + 8 significant bits: exact, down to the least bf16 value,
// which leaves 2^-133 of operands below 2^-109), and the products
// h h', (h m' + m h' + h l' + l h' + m m') are summed in two accumulators; the
// terms left out are below 2^-24 of a product, so the result is that of an
// fp32 product at six bf16 products' cost (nominal 375 TFLOP/s against 74 on
// the CUDA cores).  Infinities and NaN take part by their h alone: where the sum of
// h h' is not finite it is the result, at no cost of time.
#include <algorithm>

#include "linear.cuh"

namespace e2f {
namespace lin {

// linear_tma.cu
bool tma_operand(const void *p, long long ld);
template <bool AMN, bool BMN>
e2f_status gemm_tma(const Gemm &g, int splits, int bn, int sms, cudaStream_t s, int *rows_out);

// linear_reg.cu
template <typename T, bool AMN, bool BMN> e2f_status gemm_reg(const Gemm &g, int splits, int bn, int sms, cudaStream_t s);

// linear_skinny.cu
template <typename T> e2f_status gemm_skinny(const Gemm &g, cudaStream_t s, int *rows_out);

// linear_thin.cu
template <typename T> e2f_status gemm_thin(const Gemm &g, cudaStream_t s, int *rows_out);

// linear_small.cu
bool small_fit(int M, int N, int K, int dtype, bool tma, bool extra);
bool small_grads_fit(int M, int N, int K, int dtype);
template <typename T> e2f_status gemm_small(const Gemm &g, cudaStream_t s);
template <typename T>
e2f_status small_grads(const e2f_linear &p, const void *dz, const void *dz2, long long ldz, void *gx, long long ldgx, void *gW,
                       long long ldgw, const void *cp, int ctype, long long cld, int crows, float *gb, bool after, cudaStream_t s);

constexpr int BM = 128, BN = 128, BK = 64, NT = 256;
constexpr double ALIGN_WORK = 1 << 29;   // multiply-adds from which unaligned operands are copied first

// ---------------------------------------------------------------------------
// Partial sums of a split contraction added in a fixed order, then the
// epilogue (with no partial sums: the epilogue of zero accumulators, act'(.) dy
// = dy).  A CTA takes FROWS rows of 32 columns, a warp one of them, while there
// are few splits; else the eight warps share the splits of a row.
// ---------------------------------------------------------------------------
constexpr int FROWS = 8;
__global__ void __launch_bounds__(NT) finish_kernel(const float *__restrict__ part, int splits, int M, int N,
                                                    const __grid_constant__ Epi e) {
  __shared__ float red[NT / 32][33];
  after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.y * 32 + lane;
  const long long m0 = (long long)blockIdx.x * FROWS;
  const float bias = e.bias && n < N ? e.bias[n] : 0.f;
  float csum = 0.f;
  if (n < N) {
    const long long m = m0 + warp;
    if (m < M) {
      float v = 0.f;
#pragma unroll 8
      for (int s = 0; s < splits; ++s) v += part[((size_t)s * M + m) * N + n];
      csum = epi_elem(e, m, n, v, bias);
    }
  }
  if (e.mode == MODE_DZ && e.colpart) {
    red[warp][lane] = csum;
    __syncthreads();
    if (warp == 0 && n < N) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) s += red[w][lane];
      e.colpart[(size_t)blockIdx.x * N + n] = s;
    }
  }
}

// The same for MODE_OUT, one row and 32 columns a CTA: eight interleaved sums
// over the splits, joined in order.
__global__ void __launch_bounds__(NT) finish_row_kernel(const float *__restrict__ part, int splits, int M, int N,
                                                        const __grid_constant__ Epi e) {
  __shared__ float red[NT / 32][33];
  after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.y * 32 + lane, m = blockIdx.x;
  float v = 0.f;
  if (n < N)
#pragma unroll 8
    for (int s = warp; s < splits; s += NT / 32) v += part[((size_t)s * M + m) * N + n];
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && n < N) {
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) v += red[w][lane];
    epi_elem(e, m, n, v, e.bias ? e.bias[n] : 0.f);
  }
}

// Column sums of P rows (of dz itself, or partial ones): a CTA takes 32 columns
// and CROWS rows, 32 interleaved sums joined in order; called again on its own
// partial rows until one is left.
constexpr int CROWS = 1024;
__global__ void __launch_bounds__(1024) colsum_kernel(const void *__restrict__ p, int type, long long ld, int P, int N,
                                                      float *__restrict__ out) {
  __shared__ float red[32][33];
  after_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = blockIdx.y * 32 + lane;
  const int p0 = blockIdx.x * CROWS, p1 = min(p0 + CROWS, P);
  float s = 0.f;
  if (n < N)
#pragma unroll 8
    for (int i = p0 + w; i < p1; i += 32) s += load_as(p, type, (size_t)(i * ld) + n);
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < N) {
#pragma unroll
    for (int j = 1; j < 32; ++j) s += red[j][lane];
    out[(size_t)blockIdx.x * N + n] = s;
  }
}

// Rows of bf16 copied to a stride that is a multiple of 16 bytes: a row a warp,
// lanes along it, eight loads in flight.
__global__ void __launch_bounds__(NT) align_kernel(const __nv_bfloat16 *__restrict__ src, long long lds,
                                                   __nv_bfloat16 *__restrict__ dst, long long ldd, long long rows, int cols) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
  if (r >= rows) return;
  src += (size_t)(r * lds);
  dst += (size_t)(r * ldd);
  for (int c0 = lane; c0 < cols; c0 += 32 * U) {
    __nv_bfloat16 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 32 * u < cols) v[u] = src[c0 + 32 * u];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 32 * u < cols) dst[c0 + 32 * u] = v[u];
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int sm_count() {   // one kind of device
  static const int n = [] {
    int dev = 0, v = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    return v;
  }();
  return n;
}

// Partial rows of column sums that a MODE_DZ product leaves at most: one of eight
// rows (finish_kernel, streamed rows), of 32, or four of a 128-row tile.
static int64_t colpart_rows(int64_t M) { return (M + 7) / 8 + 4; }

template <typename T, bool AMN, bool BMN> struct Path {
  static bool tma(const Gemm &) { return false; }
  static e2f_status run_tma(const Gemm &, int, int, int, cudaStream_t, int *) { return E2F_ERR_UNSUPPORTED; }
};
template <bool AMN, bool BMN> struct Path<__nv_bfloat16, AMN, BMN> {
  static bool tma(const Gemm &g) { return tma_operand(g.A, g.lda) && tma_operand(g.B, g.ldb); }
  static e2f_status run_tma(const Gemm &g, int splits, int bn, int sms, cudaStream_t s, int *rows_out) {
    return gemm_tma<AMN, BMN>(g, splits, bn, sms, s, rows_out);
  }
};

// A product with its epilogue.  rows_out: row blocks written to e.colpart.
template <typename T, bool AMN, bool BMN>
static e2f_status run_gemm(Gemm g, cudaStream_t s, int *rows_out = nullptr) {
  const bool tma = Path<T, AMN, BMN>::tma(g);
  if constexpr (!AMN && !BMN) {
    if (g.M <= 2 || g.N <= 2) return gemm_skinny<T>(g, s, rows_out);
    if (small_fit(g.M, g.N, g.K, sizeof(T) == 4 ? E2F_F32 : E2F_BF16, tma, g.e.extra && g.N % 8 == 0)) {
      if (rows_out) *rows_out = (g.M + 31) / 32;
      return gemm_small<T>(g, s);
    }
    if (g.K <= 16 && !tma) return gemm_thin<T>(g, s, rows_out);   // (131,072 x 8 -> 512 bf16: 65 us, by TMA 44)
  }
  const int mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1) / BN, nkb = (g.K + BK - 1) / BK;
  // Fewer tiles than SMs: the contraction is split so that every SM has a
  // tile, while each split keeps four blocks; contractions of up to 15 blocks
  // stay whole (the partial sums' kernel costs more than the shorter loop
  // saves).
  const long long tiles = (long long)mt * nt;
  const int sms = sm_count();
  int splits = 1;
  if (tiles < sms && nkb >= 16) {
    splits = (int)std::min<long long>(sms / tiles, nkb / 4);
    // Operands through registers cost over a microsecond a block: further splits
    // where their rounds are shorter by more than the partial sums take (10,513 x
    // 1,427 -> 9 fp32, 83 tiles: whole 65 us, in three 48).
    if (!tma) {
      auto blocks = [&](int n) {
        const long long rounds = (tiles * n + sms - 1) / sms;
        return (double)(rounds * ((nkb + n - 1) / n)) + (n > 1 ? 3 + 2e-6 * n * g.M * g.N : 0);
      };
      const int most = std::min(8, nkb / 4);
      for (int n = splits + 1; n <= most; ++n)
        if (blocks(n) < blocks(splits)) splits = n;
    }
  }
  g.kper = (nkb + splits - 1) / splits;
  splits = (nkb + g.kper - 1) / g.kper;
  int bn = BN;
  if (tma && g.N > BN && splits == 1) {
    // TMA path: 128 x 256 tiles feed the tensor core at its full rate; 128 x
    // 128 where the wider ones would leave more of the last wave idle.
    const long long nt2 = (g.N + 2 * BN - 1) / (2 * BN);
    const long long w1 = (tiles + sms - 1) / sms, w2 = (mt * nt2 + sms - 1) / sms;
    if (9 * w2 <= 5 * w1) bn = 2 * BN;
  } else if (!tma && g.N > BN / 2 && tiles * splits * 2 <= sms) {
    bn = BN / 2;   // half the tile's latency where SMs are idle anyway
  }
  const Epi e = g.e;
  Scratch ws;
  if (splits > 1) {
    E2F_CUDA_TRY(ws.alloc(sizeof(float) * (size_t)splits * g.M * g.N, s));
    g.part = ws.as<float>();
    g.e.mode = MODE_PART;
  }
  if (rows_out) *rows_out = (g.M + (splits > 1 ? FROWS : 32) - 1) / (splits > 1 ? FROWS : 32);
  e2f_status st = tma ? Path<T, AMN, BMN>::run_tma(g, splits, bn, sms, s, rows_out)
                      : gemm_reg<T, AMN, BMN>(g, splits, bn, sms, s);
  if (st != E2F_OK || splits == 1) return st;
  const unsigned fy = (unsigned)((g.N + 31) / 32);
  if (e.mode == MODE_OUT && splits > 8) {
    E2F_LAUNCH_AFTER(finish_row_kernel, dim3((unsigned)g.M, fy), NT, 0, s, g.part, splits, g.M, g.N, e);
  } else {
    dim3 fg((unsigned)((g.M + FROWS - 1) / FROWS), fy);
    E2F_LAUNCH_AFTER(finish_kernel, fg, NT, 0, s, g.part, splits, g.M, g.N, e);
  }
  return E2F_OK;
}

// bf16 x and W on 16-byte rows for large products, which then go by TMA: there the
// copies cost less than element-wise loads in the product (100,001 x 127 -> 129
// with its gradient 239 us, 170 us so, dz in one term; below 2^29 multiply-adds it is the other
// way round).  fp32 operands pass through registers either way.  q: p with the
// copies in place of what was unaligned; after: whether a kernel was launched.
template <typename T>
static e2f_status align_operands(const e2f_linear &p, e2f_linear *q, Scratch *ws, bool *after, cudaStream_t s) {
  *q = p;
  if (sizeof(T) == 4) return E2F_OK;
  if (p.M <= 2 || p.N <= 2 || (double)p.M * p.N * p.K < ALIGN_WORK) return E2F_OK;
  auto aligned = [](const void *a, int64_t ld) {
    return ((reinterpret_cast<uintptr_t>(a) | (uintptr_t)(ld * sizeof(T))) & 15) == 0;
  };
  const bool ax = !aligned(p.x, p.ldx), aw = !aligned(p.W, p.ldw);
  if (!ax && !aw) return E2F_OK;
  constexpr int per = 16 / (int)sizeof(T);
  const int64_t ld = (p.K + per - 1) / per * per;
  const size_t xb = ax ? (sizeof(T) * (size_t)p.M * ld + 255) & ~(size_t)255 : 0, wb = aw ? sizeof(T) * (size_t)p.N * ld : 0;
  E2F_CUDA_TRY(ws->alloc(xb + wb, s));
  auto copy = [&](const void *src, int64_t lds, char *dst, int64_t rows) {
    const unsigned grid = (unsigned)((rows + NT / 32 - 1) / (NT / 32));
    E2F_LAUNCH(align_kernel, grid, NT, 0, s, static_cast<const __nv_bfloat16 *>(src), (long long)lds,
               reinterpret_cast<__nv_bfloat16 *>(dst), (long long)ld, (long long)rows, p.K);
    return E2F_OK;
  };
  if (ax) {
    const e2f_status st = copy(p.x, p.ldx, ws->as<char>(), p.M);
    if (st != E2F_OK) return st;
    q->x = ws->p;
    q->ldx = ld;
  }
  if (aw) {
    const e2f_status st = copy(p.W, p.ldw, ws->as<char>() + xb, p.N);
    if (st != E2F_OK) return st;
    q->W = ws->as<char>() + xb;
    q->ldw = ld;
  }
  *after = true;
  return E2F_OK;
}

template <typename T>
static e2f_status forward(const e2f_linear &arg, const void *res, int64_t ldr, void *out, int64_t ldo, int out_dtype,
                          cudaStream_t s) {
  Scratch copies;
  e2f_linear p;
  bool after = false;
  const e2f_status st = align_operands<T>(arg, &p, &copies, &after, s);
  if (st != E2F_OK) return st;
  Gemm g{};
  g.after = after;
  g.A = p.x; g.lda = p.ldx; g.B = p.W; g.ldb = p.ldw;
  g.M = (int)p.M; g.N = p.N; g.K = p.K;
  g.e.mode = MODE_OUT; g.e.act = p.act; g.e.bias = p.bias;
  g.e.extra = res; g.e.lde = ldr; g.e.etype = out_dtype;
  g.e.out = out; g.e.ldo = ldo; g.e.otype = out_dtype;
  return run_gemm<T, false, false>(g, s);
}

template <typename T>
static e2f_status backward(const e2f_linear &arg, const void *dy, int64_t ldg, int out_dtype, void *gx, int64_t ldgx,
                           void *gW, int64_t ldgw, float *gb, cudaStream_t s) {
  constexpr int TT = sizeof(T) == 4 ? E2F_F32 : E2F_BF16;
  const int M = (int)arg.M, N = arg.N, K = arg.K;
  if (M == 0) {   // empty sums
    if (gW) E2F_CUDA_TRY(cudaMemset2DAsync(gW, ldgw * sizeof(T), 0, K * sizeof(T), N, s));
    if (gb) E2F_CUDA_TRY(cudaMemsetAsync(gb, 0, sizeof(float) * N, s));
    return E2F_OK;
  }
  const bool prod = gx || gW;
  if (!prod && !gb) return E2F_OK;
  Scratch copies;
  e2f_linear p;
  bool after = false;
  {
    const e2f_status st = align_operands<T>(arg, &p, &copies, &after, s);
    if (st != E2F_OK) return st;
  }
  // dz: dy itself where there is no activation and the types agree
  const bool own = p.act != E2F_ACT_NONE || out_dtype != TT;
  const long long lddz = (N + 7) & ~7;
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  // (bf16: two terms, 16 bits of it.  With one, rounding dz added as much error to
  // grad_x and grad_W as rounding them: 2.35e-3 of their norm instead of 1.66e-3, for
  // which the second one costs 100,002 x 128 -> 512 125 -> 175 us, 4,099 x 1,000 ->
  // 2,050 107 -> 137.)
  const bool two = TT == E2F_BF16;
  const size_t zp = own && prod ? up(sizeof(T) * (size_t)M * lddz) : 0, zb = two ? 2 * zp : zp;
  // partial rows of the column sums, and two buffers for the sums of 1,024 rows each
  const int64_t cr = own ? colpart_rows(M) : 0, cr2 = (std::max<int64_t>(cr, M) + CROWS - 1) / CROWS;
  const size_t cb = gb ? sizeof(float) * (size_t)(cr + 2 * cr2) * N : 0;
  Scratch ws;
  if (zb + cb) E2F_CUDA_TRY(ws.alloc(zb + cb, s));
  const void *dz = dy, *dz2 = nullptr;
  long long ldz = ldg;
  // what the column sums are taken of
  const void *cp = dy;
  int ctype = out_dtype, crows = M;
  long long cld = ldg;
  if (own) {
    Gemm g{};
    g.after = after;
    g.A = p.x; g.lda = p.ldx; g.B = p.W; g.ldb = p.ldw;
    g.M = M; g.N = N; g.K = K;
    g.e.mode = MODE_DZ; g.e.act = p.act; g.e.bias = p.bias;
    g.e.extra = dy; g.e.lde = ldg; g.e.etype = out_dtype;
    g.e.out = prod ? ws.p : nullptr; g.e.out2 = prod && two ? ws.as<char>() + zp : nullptr; g.e.ldo = lddz; g.e.otype = TT;
    g.e.colpart = gb ? reinterpret_cast<float *>(ws.as<char>() + zb) : nullptr;
    crows = (int)((M + FROWS - 1) / FROWS);
    if (p.act != E2F_ACT_NONE) {
      e2f_status st = run_gemm<T, false, false>(g, s, &crows);
      if (st != E2F_OK) return st;
    } else {
      g.e.bias = nullptr;
      const dim3 grid((unsigned)((M + FROWS - 1) / FROWS), (unsigned)((N + 31) / 32));
      E2F_LIN_LAUNCH(g, finish_kernel, grid, NT, 0, s, (const float *)nullptr, 0, M, N, g.e);
    }
    after = true;
    if (prod) { dz = ws.p; dz2 = g.e.out2; ldz = lddz; }
    cp = g.e.colpart; ctype = E2F_F32; cld = N;
  }
  if (small_grads_fit(M, N, K, TT))
    return small_grads<T>(p, dz, dz2, ldz, gx, ldgx, gW, ldgw, cp, ctype, cld, crows, gb, after, s);
  if (gb) {
    float *to = reinterpret_cast<float *>(ws.as<char>() + zb) + (size_t)cr * N, *other = to + (size_t)cr2 * N;
    for (;;) {
      const int q = (crows + CROWS - 1) / CROWS;
      const dim3 grid((unsigned)q, (unsigned)((N + 31) / 32));
      if (after) E2F_LAUNCH_AFTER(colsum_kernel, grid, 1024, 0, s, cp, ctype, cld, crows, N, q == 1 ? gb : to);
      else E2F_LAUNCH(colsum_kernel, grid, 1024, 0, s, cp, ctype, cld, crows, N, q == 1 ? gb : to);
      after = true;
      if (q == 1) break;
      cp = to; ctype = E2F_F32; cld = N; crows = q;
      std::swap(to, other);
    }
  }
  if (gx) {
    Gemm g{};
    g.A = dz; g.A2 = dz2; g.lda = ldz; g.B = p.W; g.ldb = p.ldw;
    g.M = M; g.N = K; g.K = N;
    g.after = after;
    after = true;
    g.e.mode = MODE_OUT; g.e.act = E2F_ACT_NONE;
    g.e.out = gx; g.e.ldo = ldgx; g.e.otype = TT;
    e2f_status st = run_gemm<T, false, true>(g, s);
    if (st != E2F_OK) return st;
  }
  if (gW) {
    Gemm g{};
    g.A = dz; g.A2 = dz2; g.lda = ldz; g.B = p.x; g.ldb = p.ldx;
    g.M = N; g.N = K; g.K = M;
    g.after = after;
    g.e.mode = MODE_OUT; g.e.act = E2F_ACT_NONE;
    g.e.out = gW; g.e.ldo = ldgw; g.e.otype = TT;
    e2f_status st = run_gemm<T, true, true>(g, s);
    if (st != E2F_OK) return st;
  }
  return E2F_OK;
}

}  // namespace lin

e2f_status linear_forward_impl(const e2f_linear *p, const void *residual, int64_t ldr, void *out, int64_t ldo,
                               int out_dtype, cudaStream_t s) {
  return p->dtype == E2F_F32 ? lin::forward<float>(*p, residual, ldr, out, ldo, out_dtype, s)
                             : lin::forward<__nv_bfloat16>(*p, residual, ldr, out, ldo, out_dtype, s);
}

e2f_status linear_backward_impl(const e2f_linear *p, const void *grad_out, int64_t ldg, int out_dtype, void *grad_x,
                                int64_t ldgx, void *grad_W, int64_t ldgw, float *grad_bias, cudaStream_t s) {
  return p->dtype == E2F_F32
             ? lin::backward<float>(*p, grad_out, ldg, out_dtype, grad_x, ldgx, grad_W, ldgw, grad_bias, s)
             : lin::backward<__nv_bfloat16>(*p, grad_out, ldg, out_dtype, grad_x, ldgx, grad_W, ldgw, grad_bias, s);
}

}  // namespace e2f
