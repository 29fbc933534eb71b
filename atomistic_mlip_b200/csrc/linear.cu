// Linear layers with bias, activation and residual in the epilogue, and their
// gradient:
//
//   forward    y  = act(x W^T + b) + r
//   backward   z  = x W^T + b (formed again: nothing but y leaves the forward),
//              dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
//
// All products run on the tensor cores.  bf16 operands are used as they are,
// fp32 accumulation.  fp32 operands are split into three bf16 terms each,
// x = h + m + l (8 + 8 + 8 significant bits: exact), and the products
// h h', (h m' + m h' + h l' + l h' + m m') are summed in two accumulators; the
// terms left out are below 2^-24 of a product, so the result is that of an
// fp32 product at six bf16 products' cost (nominal 375 TFLOP/s against 74 on
// the CUDA cores).  A product that meets an infinity gives NaN in the split
// form (inf * 0); such elements are summed again from the fp32 operands.
#include <algorithm>

#include "linear.cuh"

namespace e2f {
namespace lin {

// linear_tma.cu
bool tma_operand(const void *p, long long ld);
template <bool AMN, bool BMN> e2f_status gemm_tma(const Gemm &g, int splits, int bn, int sms, cudaStream_t s);

constexpr int BM = 128, BN = 128, BK = 64, NT = 256;
constexpr int TILE_BYTES = 128 * BK * 2;     // one 128 x 64 bf16 operand tile
constexpr int EPITCH = BN + 1;               // accumulator tile in shared memory, floats per row

// ---------------------------------------------------------------------------
// operand tiles: 128 x 64 bf16 in 128-byte swizzled rows.  K-major: a row
// holds 64 k.  MN-major: two blocks of 64 m, a row holds the 64 m of one k.
// ---------------------------------------------------------------------------
template <bool MN> __device__ __forceinline__ uint32_t chunk_off(int q) {
  if (!MN) {   // chunk of 8 k
    const int r = q >> 3, c = q & 7;
    return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  }
  const int k = q >> 4, c = q & 15;   // chunk of 8 m
  return (uint32_t)((c >> 3) * 8192 + k * 128 + (((c & 7) ^ (k & 7)) << 4));
}

// Descriptor of such a tile from the k-th (multiple of 16) column on: 128-byte
// swizzle, 1024 bytes from eight rows to the next; MN-major: 8192 bytes from
// one block of 64 m to the next.
template <bool MN> __device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, int k) {
  const uint32_t a = saddr + (MN ? k * 128 : k * 2);
  return tc::smem_desc(a, MN ? 8192 : 16, 1024) | (uint64_t)2 << 61;
}

// Eight consecutive elements of an operand; nv of them are inside.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { uint4 a; };
template <> struct Raw<float> { float4 a, b; };

__device__ __forceinline__ void load8(Raw<__nv_bfloat16> &r, const __nv_bfloat16 *p, int nv, bool vec) {
  if (vec && nv >= 8) {
    r.a = __ldg(reinterpret_cast<const uint4 *>(p));
    return;
  }
  const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < nv ? __ldg(u + 2 * i) : 0u, hi = 2 * i + 1 < nv ? __ldg(u + 2 * i + 1) : 0u;
    w[i] = lo | hi << 16;
  }
  r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(Raw<float> &r, const float *p, int nv, bool vec) {
  if (vec && nv >= 8) {
    r.a = __ldg(reinterpret_cast<const float4 *>(p));
    r.b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    return;
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < nv ? __ldg(p + i) : 0.f;
  r.a = make_float4(v[0], v[1], v[2], v[3]);
  r.b = make_float4(v[4], v[5], v[6], v[7]);
}

// Terms of a chunk to shared memory, TILE_BYTES apart.
__device__ __forceinline__ void put8(const Raw<__nv_bfloat16> &r, uint8_t *p) { *reinterpret_cast<uint4 *>(p) = r.a; }
__device__ __forceinline__ void split2(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l) {
  h = pack_bf16x2(x, y);
  x -= __uint_as_float(h << 16);
  y -= __uint_as_float(h & 0xffff0000u);
  m = pack_bf16x2(x, y);
  x -= __uint_as_float(m << 16);
  y -= __uint_as_float(m & 0xffff0000u);
  l = pack_bf16x2(x, y);
}
__device__ __forceinline__ void put8(const Raw<float> &r, uint8_t *p) {
  uint4 h, m, l;
  split2(r.a.x, r.a.y, h.x, m.x, l.x);
  split2(r.a.z, r.a.w, h.y, m.y, l.y);
  split2(r.b.x, r.b.y, h.z, m.z, l.z);
  split2(r.b.z, r.b.w, h.w, m.w, l.w);
  *reinterpret_cast<uint4 *>(p) = h;
  *reinterpret_cast<uint4 *>(p + TILE_BYTES) = m;
  *reinterpret_cast<uint4 *>(p + 2 * TILE_BYTES) = l;
}

// The chunks of one operand tile this thread carries: rows r0.. (m or n),
// contraction k0..; RN rows and KN columns exist.
template <typename T, bool MN>
__device__ __forceinline__ void fetch_tile(Raw<T> (&r)[4], const T *P, long long ld, int r0, int RN, int k0, int KN,
                                           bool vec) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int q = threadIdx.x + NT * j;
    const int row = MN ? k0 + (q >> 4) : r0 + (q >> 3);          // strided index
    const int col = MN ? r0 + 8 * (q & 15) : k0 + 8 * (q & 7);   // contiguous index
    const int nrow = MN ? KN : RN, ncol = MN ? RN : KN;
    const int nv = row < nrow ? ncol - col : 0;
    load8(r[j], P + (nv > 0 ? (size_t)((long long)row * ld) + col : 0), nv, vec);
  }
}
template <typename T, bool MN> __device__ __forceinline__ void put_tile(const Raw<T> (&r)[4], uint8_t *s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) put8(r[j], s + chunk_off<MN>(threadIdx.x + NT * j));
}

// An element of the product from the fp32 operands themselves.
template <bool AMN, bool BMN>
__device__ __noinline__ float dot_again(const Gemm &g, int m, int n, int k0, int k1) {
  const float *A = static_cast<const float *>(g.A), *B = static_cast<const float *>(g.B);
  float s = 0.f;
  for (int k = k0; k < k1; ++k)
    s = fmaf(AMN ? A[(size_t)(k * g.lda) + m] : A[(size_t)(m * g.lda) + k],
             BMN ? B[(size_t)(k * g.ldb) + n] : B[(size_t)(n * g.ldb) + k], s);
  return s;
}

// ---------------------------------------------------------------------------
// One 128 x 128 output tile per CTA (blockIdx: row tile, column tile, split of
// the contraction).  All threads carry the operands global -> registers ->
// shared memory (any stride and alignment; the fp32 form splits on the way),
// two stages; the next block's loads are in flight while the tensor core works.
// ---------------------------------------------------------------------------
template <typename T> constexpr int terms() { return sizeof(T) == 4 ? 3 : 1; }
template <typename T> constexpr size_t staged_smem() {
  const size_t ops = 2 * (size_t)terms<T>() * 2 * TILE_BYTES, acc = sizeof(float) * BM * EPITCH;
  return (ops > acc ? ops : acc) + 1024;
}

template <typename T, bool AMN, bool BMN>
__global__ void __launch_bounds__(NT, 1) gemm_staged_kernel(const __grid_constant__ Gemm g, int *err) {
  using namespace tc;
  constexpr int NS = terms<T>();
  constexpr int OP = NS * TILE_BYTES;          // one operand of a stage
  constexpr uint32_t TCOLS = NS == 3 ? 256 : 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t bar[2];
  __shared__ uint32_t tslot;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) { mbar_init(&bar[0], 1); mbar_init(&bar[1], 1); mbar_fence_init(); }
  __syncthreads();
  if (warp == 0) { tmem_alloc(&tslot, TCOLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tslot;
  const int m0 = blockIdx.x * BM, n0 = blockIdx.y * BN;
  const int nkb = (g.K + BK - 1) / BK;
  const int kb0 = blockIdx.z * g.kper, kb1 = kb0 + g.kper < nkb ? kb0 + g.kper : nkb;
  const T *A = static_cast<const T *>(g.A), *B = static_cast<const T *>(g.B);
  const bool va = ((reinterpret_cast<uintptr_t>(A) | (uintptr_t)(g.lda * sizeof(T))) & 15) == 0;
  const bool vb = ((reinterpret_cast<uintptr_t>(B) | (uintptr_t)(g.ldb * sizeof(T))) & 15) == 0;
  const int nb = g.N - n0 < BN ? (g.N - n0 + 15) & ~15 : BN;   // columns the tensor core works on
  const uint32_t id = idesc_bf16(128, nb, AMN, BMN);
  Raw<T> ra[4], rb[4];
  bool dead = false;
  fetch_tile<T, AMN>(ra, A, g.lda, m0, g.M, kb0 * BK, g.K, va);
  fetch_tile<T, BMN>(rb, B, g.ldb, n0, g.N, kb0 * BK, g.K, vb);
  for (int kb = kb0; kb < kb1; ++kb) {
    const int i = kb - kb0, st = i & 1;
    uint8_t *sA = smem + st * 2 * OP, *sB = sA + OP;
    if (i >= 2) {   // the products that read this stage two blocks ago are done
      const bool ok = mbar_wait(&bar[st], ((i >> 1) - 1) & 1, 1u << 26);
      dead = __syncthreads_or(!ok) != 0;
      if (dead) break;
    }
    put_tile<T, AMN>(ra, sA);
    put_tile<T, BMN>(rb, sB);
    fence_async_smem();
    __syncthreads();
    if (t == 0) {
      tc_fence_after();
      const uint32_t a0 = smem_addr(sA), b0 = smem_addr(sB);
#pragma unroll
      for (int k = 0; k < BK; k += 16) {
        const uint32_t first = i > 0 || k > 0 ? 1u : 0u;
        mma_bf16_ss(tb, tile_desc<AMN>(a0, k), tile_desc<BMN>(b0, k), id, first);
        if (NS == 3) {
          const uint32_t am = a0 + TILE_BYTES, al = am + TILE_BYTES, bm = b0 + TILE_BYTES, bl = bm + TILE_BYTES;
          mma_bf16_ss(tb + 128, tile_desc<AMN>(a0, k), tile_desc<BMN>(bl, k), id, first);
          mma_bf16_ss(tb + 128, tile_desc<AMN>(al, k), tile_desc<BMN>(b0, k), id, 1u);
          mma_bf16_ss(tb + 128, tile_desc<AMN>(am, k), tile_desc<BMN>(bm, k), id, 1u);
          mma_bf16_ss(tb + 128, tile_desc<AMN>(a0, k), tile_desc<BMN>(bm, k), id, 1u);
          mma_bf16_ss(tb + 128, tile_desc<AMN>(am, k), tile_desc<BMN>(b0, k), id, 1u);
        }
      }
      mma_commit(&bar[st]);
    }
    if (kb + 1 < kb1) {
      fetch_tile<T, AMN>(ra, A, g.lda, m0, g.M, (kb + 1) * BK, g.K, va);
      fetch_tile<T, BMN>(rb, B, g.ldb, n0, g.N, (kb + 1) * BK, g.K, vb);
    }
  }
  const int nblk = kb1 - kb0;
  if (!dead) {   // a commit covers every product issued before it
    const bool ok = mbar_wait(&bar[(nblk - 1) & 1], ((nblk - 1) >> 1) & 1, 1u << 26);
    dead = __syncthreads_or(!ok) != 0;
  }
  if (dead) {
    if (t == 0) atomicExch(err, E2F_ERR_TIMEOUT);
  } else {
    // accumulators -> shared memory (the operand stages are done with) -> rows
    tc_fence_after();
    float *acc = reinterpret_cast<float *>(smem);
    {
      const int row = 32 * (warp & 3) + lane, c0 = 64 * (warp >> 2);
      const uint32_t ta = tb + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        if (c0 + c < nb) {
          float v[16], w[16];
          if (NS == 3) tmem_ld_32x32b_x16x2(ta + c0 + c, ta + 128 + c0 + c, v, w);
          else tmem_ld_32x32b_x16(ta + c0 + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[row * EPITCH + c0 + c + j] = NS == 3 ? v[j] + w[j] : v[j];
        }
      }
    }
    __syncthreads();
    float bias[4], csum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + lane + 32 * j;
      bias[j] = g.e.mode != MODE_PART && g.e.bias && n < g.N ? g.e.bias[n] : 0.f;
      csum[j] = 0.f;
    }
    for (int r = warp; r < BM && m0 + r < g.M; r += NT / 32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + lane + 32 * j;
        if (n < g.N) {
          float v = acc[r * EPITCH + lane + 32 * j];
          if (NS == 3 && v != v) v = dot_again<AMN, BMN>(g, m0 + r, n, kb0 * BK, min(kb1 * BK, g.K));
          if (g.e.mode == MODE_PART) g.part[((size_t)blockIdx.z * g.M + m0 + r) * g.N + n] = v;
          else csum[j] += epi_elem(g.e, m0 + r, n, v, bias[j]);
        }
      }
    }
    if (g.e.mode == MODE_DZ && g.e.colpart) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[warp * BN + lane + 32 * j] = csum[j];
      __syncthreads();
      if (t < BN && n0 + t < g.N) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) s += acc[w * BN + t];
        g.e.colpart[(size_t)blockIdx.x * g.N + n0 + t] = s;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, TCOLS);
}

// ---------------------------------------------------------------------------
// Partial sums of a split contraction added in a fixed order, then the
// epilogue (with no partial sums: the epilogue of zero accumulators, act'(.) dy
// = dy).  A CTA takes FROWS rows of 32 columns; a warp takes whole rows (one
// element a lane) while there are few splits, else the eight warps share the
// splits of a row.
// ---------------------------------------------------------------------------
constexpr int FROWS = 32;
__global__ void __launch_bounds__(NT) finish_kernel(const float *__restrict__ part, int splits, int M, int N,
                                                    const __grid_constant__ Epi e) {
  __shared__ float red[NT / 32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.y * 32 + lane;
  const long long m0 = (long long)blockIdx.x * FROWS;
  const float bias = e.bias && n < N ? e.bias[n] : 0.f;
  float csum = 0.f;
  if (n < N) {
#pragma unroll
    for (int r = 0; r < FROWS / 8; ++r) {
      const long long m = m0 + warp + 8 * r;
      if (m >= M) break;
      float v = 0.f;
#pragma unroll 8
      for (int s = 0; s < splits; ++s) v += part[((size_t)s * M + m) * N + n];
      csum += epi_elem(e, m, n, v, bias);
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

// Column sums of P partial rows: a CTA takes 32 columns and CROWS rows, eight
// interleaved sums joined in order; called again on its own partial rows until
// one is left.
constexpr int CROWS = 128;
__global__ void __launch_bounds__(256) colsum_kernel(const float *__restrict__ part, int P, int N, float *__restrict__ out) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = blockIdx.x * 32 + lane;
  const int p0 = blockIdx.y * CROWS, p1 = min(p0 + CROWS, P);
  float s = 0.f;
  if (n < N)
#pragma unroll 8
    for (int p = p0 + w; p < p1; p += 8) s += part[(size_t)p * N + n];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < N) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += red[j][lane];
    out[(size_t)blockIdx.y * N + n] = s;
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

template <typename T, bool AMN, bool BMN> static e2f_status launch_staged(const Gemm &g, dim3 grid, cudaStream_t s) {
  int *err = device_error_flag();
  if (!err) return E2F_ERR_CUDA;
  constexpr auto k = gemm_staged_kernel<T, AMN, BMN>;
  E2F_CUDA_TRY(allow_smem<k>(staged_smem<T>()));
  E2F_LAUNCH(k, grid, NT, staged_smem<T>(), s, g, err);
  return E2F_OK;
}

// Row blocks whose column sums a MODE_DZ product leaves (upper bound).
static int64_t colpart_rows(int64_t M) { return (M + FROWS - 1) / FROWS; }

template <typename T, bool AMN, bool BMN> struct Path {
  static bool tma(const Gemm &) { return false; }
  static e2f_status run_tma(const Gemm &, int, int, int, cudaStream_t) { return E2F_ERR_UNSUPPORTED; }
};
template <bool AMN, bool BMN> struct Path<__nv_bfloat16, AMN, BMN> {
  static bool tma(const Gemm &g) { return tma_operand(g.A, g.lda) && tma_operand(g.B, g.ldb); }
  static e2f_status run_tma(const Gemm &g, int splits, int bn, int sms, cudaStream_t s) {
    return gemm_tma<AMN, BMN>(g, splits, bn, sms, s);
  }
};

// A product with its epilogue.  rows_out: row blocks written to e.colpart.
template <typename T, bool AMN, bool BMN>
static e2f_status run_gemm(Gemm g, cudaStream_t s, int *rows_out = nullptr) {
  const int mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1) / BN, nkb = (g.K + BK - 1) / BK;
  if (nt > 65535) return E2F_ERR_UNSUPPORTED;
  // Fewer tiles than SMs: the contraction is split so that every SM has a
  // tile, while each split keeps four blocks (below that the partial sums cost
  // more than the shorter loop saves).
  const long long tiles = (long long)mt * nt;
  const int sms = sm_count();
  int splits = 1;
  if (tiles < sms && nkb >= 8) splits = (int)std::min<long long>(sms / tiles, nkb / 4);
  g.kper = (nkb + splits - 1) / splits;
  splits = (nkb + g.kper - 1) / g.kper;
  const bool tma = Path<T, AMN, BMN>::tma(g);
  // TMA path: 128 x 256 tiles feed the tensor core at its full rate; 128 x 128
  // where the wider ones would leave more of the last wave idle.
  int bn = BN;
  if (tma && g.N > BN && splits == 1) {
    const long long nt2 = (g.N + 2 * BN - 1) / (2 * BN);
    const long long w1 = (tiles + sms - 1) / sms, w2 = (mt * nt2 + sms - 1) / sms;
    if (9 * w2 <= 5 * w1) bn = 2 * BN;
  }
  const Epi e = g.e;
  Scratch ws;
  if (splits > 1) {
    E2F_CUDA_TRY(ws.alloc(sizeof(float) * (size_t)splits * g.M * g.N, s));
    g.part = ws.as<float>();
    g.e.mode = MODE_PART;
  }
  e2f_status st = tma ? Path<T, AMN, BMN>::run_tma(g, splits, bn, sms, s)
                      : launch_staged<T, AMN, BMN>(g, dim3(mt, nt, splits), s);
  if (rows_out) *rows_out = tma || splits > 1 ? (int)colpart_rows(g.M) : mt;
  if (st != E2F_OK || splits == 1) return st;
  const unsigned fy = (unsigned)((g.N + 31) / 32);
  if (e.mode == MODE_OUT && splits > 8) {
    E2F_LAUNCH(finish_row_kernel, dim3((unsigned)g.M, fy), NT, 0, s, g.part, splits, g.M, g.N, e);
  } else {
    dim3 fg((unsigned)((g.M + FROWS - 1) / FROWS), fy);
    E2F_LAUNCH(finish_kernel, fg, NT, 0, s, g.part, splits, g.M, g.N, e);
  }
  return E2F_OK;
}

template <typename T>
static e2f_status forward(const e2f_linear &p, const void *res, int64_t ldr, void *out, int64_t ldo, int out_dtype,
                          cudaStream_t s) {
  Gemm g{};
  g.A = p.x; g.lda = p.ldx; g.B = p.W; g.ldb = p.ldw;
  g.M = (int)p.M; g.N = p.N; g.K = p.K;
  g.e.mode = MODE_OUT; g.e.act = p.act; g.e.bias = p.bias;
  g.e.extra = res; g.e.lde = ldr; g.e.etype = out_dtype;
  g.e.out = out; g.e.ldo = ldo; g.e.otype = out_dtype;
  return run_gemm<T, false, false>(g, s);
}

template <typename T>
static e2f_status backward(const e2f_linear &p, const void *dy, int64_t ldg, int out_dtype, void *gx, int64_t ldgx,
                           void *gW, int64_t ldgw, float *gb, cudaStream_t s) {
  constexpr int TT = sizeof(T) == 4 ? E2F_F32 : E2F_BF16;
  const int M = (int)p.M, N = p.N, K = p.K;
  if (M == 0) {   // empty sums
    if (gW) E2F_CUDA_TRY(cudaMemset2DAsync(gW, ldgw * sizeof(T), 0, K * sizeof(T), N, s));
    if (gb) E2F_CUDA_TRY(cudaMemsetAsync(gb, 0, sizeof(float) * N, s));
    return E2F_OK;
  }
  const bool prod = gx || gW;
  if (!prod && !gb) return E2F_OK;
  // dz: dy itself where there is no activation and the types agree
  const bool own = p.act != E2F_ACT_NONE || out_dtype != TT;
  const long long lddz = (N + 7) & ~7;
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  const size_t zb = own && prod ? up(sizeof(T) * (size_t)M * lddz) : 0;
  // partial rows of the column sums, and one level of their sums
  const int64_t cr = colpart_rows(M);
  const size_t cb = gb ? sizeof(float) * (size_t)(cr + (cr + CROWS - 1) / CROWS) * N : 0;
  Scratch ws;
  if (zb + cb) E2F_CUDA_TRY(ws.alloc(zb + cb, s));
  const void *dz = dy;
  long long ldz = ldg;
  int crows = 0;
  if (own || gb) {
    Gemm g{};
    g.A = p.x; g.lda = p.ldx; g.B = p.W; g.ldb = p.ldw;
    g.M = M; g.N = N; g.K = K;
    g.e.mode = MODE_DZ; g.e.act = p.act; g.e.bias = p.bias;
    g.e.extra = dy; g.e.lde = ldg; g.e.etype = out_dtype;
    g.e.out = own && prod ? ws.p : nullptr; g.e.ldo = lddz; g.e.otype = TT;
    g.e.colpart = gb ? reinterpret_cast<float *>(ws.as<char>() + zb) : nullptr;
    if (p.act != E2F_ACT_NONE) {
      e2f_status st = run_gemm<T, false, false>(g, s, &crows);
      if (st != E2F_OK) return st;
    } else {
      dim3 fg((unsigned)((M + FROWS - 1) / FROWS), (unsigned)((N + 31) / 32));
      g.e.bias = nullptr;
      E2F_LAUNCH(finish_kernel, fg, NT, 0, s, nullptr, 0, M, N, g.e);
      crows = (int)fg.x;
    }
    if (own && prod) { dz = ws.p; ldz = lddz; }
    if (gb) {
      float *from = g.e.colpart, *to = from + (size_t)cr * N;
      for (int P = crows;; std::swap(from, to)) {
        const int q = (P + CROWS - 1) / CROWS;
        E2F_LAUNCH(colsum_kernel, dim3((N + 31) / 32, q), 256, 0, s, from, P, N, q == 1 ? gb : to);
        if ((P = q) == 1) break;
      }
    }
  }
  if (gx) {
    Gemm g{};
    g.A = dz; g.lda = ldz; g.B = p.W; g.ldb = p.ldw;
    g.M = M; g.N = K; g.K = N;
    g.e.mode = MODE_OUT; g.e.act = E2F_ACT_NONE;
    g.e.out = gx; g.e.ldo = ldgx; g.e.otype = TT;
    e2f_status st = run_gemm<T, false, true>(g, s);
    if (st != E2F_OK) return st;
  }
  if (gW) {
    Gemm g{};
    g.A = dz; g.lda = ldz; g.B = p.x; g.ldb = p.ldx;
    g.M = N; g.N = K; g.K = M;
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
