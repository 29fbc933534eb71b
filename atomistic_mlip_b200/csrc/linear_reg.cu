// Products of the linear layers whose operands go through registers: fp32
// operands, which are split into bf16 terms on the way, and bf16 operands whose
// rows do not start on 16-byte boundaries.  Any stride and alignment.
//
// A persistent CTA per SM walks output tiles of 128 x bn (bn = 128 or 64).
// Warps 0-15 carry the operands, 64 contraction columns a stage: global loads
// of the next stage are in flight while this one is split and written to shared
// memory (128-byte swizzle) and multiplied; warp 16 issues the MMAs into one of
// two accumulators (fp32 operands: two of 128 columns each, see linear.cu);
// warps 20-27 run the epilogue of the other one meanwhile.  One stage of fp32
// operands costs the tensor core 24 MMAs of 64 cycles and shared memory 96 KB
// written and 192 KB read (2,304 cycles): shared memory bounds it, at 265
// TFLOP/s nominal.
// Measured (fp32): 4,096 x 4,096 -> 2,048 410 us, 168 TFLOP/s; 100,002 x 128 -> 512
// 125 us, with SiLU 140; 10,304 x 128 -> 128 10 us, all of it latency.
#include <algorithm>

#include "linear_epi.cuh"

namespace e2f {
namespace lin {
namespace reg {

constexpr int BM = 128, BK = 64;
constexpr int CONV = 512, CTRL_WARP = 16, EPI_WARP = 20, NT = 896, LAUNCH_REGS = 72;
constexpr int TILE_BYTES = 128 * BK * 2;     // one 128 x 64 bf16 operand tile
template <typename T> constexpr int terms() { return sizeof(T) == 4 ? 3 : 1; }
template <typename T> constexpr int stages() { return sizeof(T) == 4 ? 2 : 4; }
// NA: terms of A in memory, each bf16, multiplied with B one after the other (dz of
// the bf16 backward; 1 for all else)
template <typename T, int NA> constexpr int ring() { return stages<T>() * (NA + 1) * terms<T>() * TILE_BYTES; }
constexpr int STAGING = 8 * 32 * 32 * 4, SBIAS = 8 * 32 * 4;
template <typename T, int NA> constexpr size_t smem_bytes() { return ring<T, NA>() + STAGING + SBIAS + 256 + 1024; }

struct Args {
  Gemm g;
  Sched s;
  int *err;
};

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
// The terms of half the value: the largest fp32 values do not round to a bf16
// infinity so.  (4,096 x 4,096 -> 2,048: 405 us without the halving, 409 with it, 440
// if they are told apart instead.)  Infinities and NaN have themselves as h; their m
// and l are NaN, which join() below leaves out.
constexpr float SPLIT_SCALE = 4.f;   // of a product of two such sums
__device__ __forceinline__ void split2(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l) {
  const f2 half = mul2({x, y}, both(0.5f));
  x = half.x;
  y = half.y;
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

// The sum of h h' and that of the smaller products.  Where the first is not
// finite it is the result: the infinities and NaN of the operands are in it as in an
// fp32 product.
__device__ __forceinline__ float join(float hh, float small) { return fabsf(hh) < INFINITY ? hh + small : hh; }

// The chunks of one operand tile this thread carries: rows r0 .. (m or n) below
// RN, contraction k0 .. below KN.
template <typename T, bool MN>
__device__ __forceinline__ void fetch_tile(Raw<T> (&r)[2], const T *P, long long ld, int r0, int RN, int k0, int KN, bool vec) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int q = threadIdx.x + CONV * j;
    const int row = MN ? k0 + (q >> 4) : r0 + (q >> 3);          // strided index
    const int col = MN ? r0 + 8 * (q & 15) : k0 + 8 * (q & 7);   // contiguous index
    const int nv = row < (MN ? KN : RN) ? (MN ? RN : KN) - col : 0;
    load8(r[j], P + (nv > 0 ? (size_t)((long long)row * ld) + col : 0), nv, vec);
  }
}
// ... to the stage; rows from nb on are not multiplied.
template <typename T, bool MN> __device__ __forceinline__ void put_tile(const Raw<T> (&r)[2], uint8_t *s, int nb) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int q = threadIdx.x + CONV * j;
    if ((MN ? 8 * (q & 15) : q >> 3) < nb) put8(r[j], s + chunk_off<MN>(q));
  }
}

// Registers: 16 carrying warps 64, four control warps 24, eight epilogue warps
// 112 of the 72 a thread the block is launched with: 4 * 64 + 24 + 2 * 112 = 7 * 72.
template <typename T, bool AMN, bool BMN, int EPI, bool LONGK, int NA>
__global__ void __launch_bounds__(NT, 1) gemm_reg_kernel(const __grid_constant__ Args a) {
  using namespace tc;
  constexpr int NS = terms<T>(), ST = stages<T>(), OP = NS * TILE_BYTES, RING = ring<T, NA>();
  constexpr int OA = NA * OP, SB = OA + OP;   // A's part of a stage, the stage
  constexpr int ACC = NS == 3 ? 256 : 128;   // TMEM columns of an accumulator
  constexpr uint32_t LIMIT = 1u << 26;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float *staging = reinterpret_cast<float *>(smem + RING);
  float *sbiases = staging + STAGING / 4;
  uint64_t *full = reinterpret_cast<uint64_t *>(sbiases + SBIAS / 4), *empty = full + ST, *tfull = empty + ST,
           *tempty = tfull + 2;
  __shared__ uint32_t tslot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&full[i], CONV / 32); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&tfull[i], 1); mbar_init(&tempty[i], 8); }
    mbar_fence_init();
  }
  __syncthreads();
  if (warp == CTRL_WARP) { tmem_alloc(&tslot, 2 * ACC); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot;
  const Gemm &g = a.g;
  after_previous();

  if (warp < CTRL_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const T *A = static_cast<const T *>(g.A), *A2 = static_cast<const T *>(g.A2), *B = static_cast<const T *>(g.B);
    const bool va = ((reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(A2) | (uintptr_t)(g.lda * sizeof(T))) & 15) == 0;
    const bool vb = ((reinterpret_cast<uintptr_t>(B) | (uintptr_t)(g.ldb * sizeof(T))) & 15) == 0;
    Raw<T> ra[2], ra2[2], rb[2];
    int i = blockIdx.x, s = 0;
    uint32_t ph = 1;   // the first pass over the ring finds it empty
    bool ok = true;
    if (i < a.s.tiles) {
      Tile t = tile_of(g, a.s, i);
      int kb = t.kb0;
      fetch_tile<T, AMN>(ra, A, g.lda, t.m0, g.M, kb * BK, g.K, va);
      if (NA == 2) fetch_tile<T, AMN>(ra2, A2, g.lda, t.m0, g.M, kb * BK, g.K, va);
      fetch_tile<T, BMN>(rb, B, g.ldb, t.n0, min(g.N, t.n0 + a.s.bn), kb * BK, g.K, vb);
      while (true) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph, LIMIT));
        if (!ok) break;
        uint8_t *sA = smem + s * SB;
        put_tile<T, AMN>(ra, sA, BM);
        if (NA == 2) put_tile<T, AMN>(ra2, sA + OP, BM);
        put_tile<T, BMN>(rb, sA + OA, min(a.s.bn, (g.N - t.n0 + 15) & ~15));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == ST) { s = 0; ph ^= 1; }
        if (++kb == t.kb1) {
          i += gridDim.x;
          if (i >= a.s.tiles) break;
          t = tile_of(g, a.s, i);
          kb = t.kb0;
        }
        fetch_tile<T, AMN>(ra, A, g.lda, t.m0, g.M, kb * BK, g.K, va);
        if (NA == 2) fetch_tile<T, AMN>(ra2, A2, g.lda, t.m0, g.M, kb * BK, g.K, va);
        fetch_tile<T, BMN>(rb, B, g.ldb, t.n0, min(g.N, t.n0 + a.s.bn), kb * BK, g.K, vb);
      }
    }
    if (!ok && lane == 0) atomicExch(a.err, E2F_ERR_TIMEOUT);
  } else if (warp < EPI_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
    if (warp == CTRL_WARP && lane == 0) {
      int s = 0, u = 0;   // ring slot, accumulators issued
      uint32_t ph = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < a.s.tiles && ok; i += gridDim.x) {
        const Tile t = tile_of(g, a.s, i);
        const uint32_t id = idesc_bf16(128, min(a.s.bn, (g.N - t.n0 + 15) & ~15), AMN, BMN);
        for (int kc = t.kb0; kc < t.kb1 && ok; kc += LONGK ? KCHUNK : t.kb1 - t.kb0, ++u) {
          const int ke = LONGK ? min(kc + KCHUNK, t.kb1) : t.kb1;
          const uint32_t acc = tmem + (u & 1) * ACC;
          ok = mbar_wait(&tempty[u & 1], ((u >> 1) & 1) ^ 1, LIMIT);
          if (!ok) break;
          tc_fence_after();
          for (int kb = kc; kb < ke; ++kb) {
            ok = mbar_wait(&full[s], ph, LIMIT);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a0 = smem_addr(smem + s * SB), b0 = a0 + OA;
#pragma unroll
            for (int k = 0; k < BK; k += 16) {
              const uint32_t more = kb > kc || k > 0 ? 1u : 0u;
              mma_bf16_ss(acc, tile_desc<AMN>(a0, k), tile_desc<BMN>(b0, k), id, more);
              if (NA == 2) mma_bf16_ss(acc, tile_desc<AMN>(a0 + OP, k), tile_desc<BMN>(b0, k), id, 1u);
              if (NS == 3) {
                const uint32_t am = a0 + TILE_BYTES, al = am + TILE_BYTES, bm = b0 + TILE_BYTES, bl = bm + TILE_BYTES;
                mma_bf16_ss(acc + 128, tile_desc<AMN>(a0, k), tile_desc<BMN>(bl, k), id, more);
                mma_bf16_ss(acc + 128, tile_desc<AMN>(al, k), tile_desc<BMN>(b0, k), id, 1u);
                mma_bf16_ss(acc + 128, tile_desc<AMN>(am, k), tile_desc<BMN>(bm, k), id, 1u);
                mma_bf16_ss(acc + 128, tile_desc<AMN>(a0, k), tile_desc<BMN>(bm, k), id, 1u);
                mma_bf16_ss(acc + 128, tile_desc<AMN>(am, k), tile_desc<BMN>(b0, k), id, 1u);
              }
            }
            mma_commit(&empty[s]);
            if (++s == ST) { s = 0; ph ^= 1; }
          }
          mma_commit(&tfull[u & 1]);
        }
      }
      if (!ok) atomicExch(a.err, E2F_ERR_TIMEOUT);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    const int ew = warp - EPI_WARP, quarter = warp & 3, half = ew >> 2;   // chunks of 32 columns: half, half + 2
    const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
    float *st = staging + ew * 32 * 32;
    float *sbias = sbiases + ew * 32;
    const Epi &e = g.e;
    constexpr bool EXTRA = EPI >= RES;
    int u = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < a.s.tiles && ok; i += gridDim.x) {
      const Tile t = tile_of(g, a.s, i);
      const int mw = t.m0 + 32 * quarter;
      const Rows rw = rows_of(g, t.split, mw, lane);
      float bias[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = t.n0 + 32 * (half + 2 * c) + lane;
        bias[c] = EPI != PLAIN && e.bias && n < g.N ? __ldg(e.bias + n) : 0.f;
      }
      float acc[LONGK ? 64 : 1];
      if (LONGK) {
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0.f;
      }
      for (int kc = t.kb0; kc < t.kb1; kc += LONGK ? KCHUNK : t.kb1 - t.kb0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[u & 1], (u >> 1) & 1, LIMIT));
        if (!ok) break;
        tc_fence_after();
        if (LONGK) {
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float v[16];
            const uint32_t ta = tq + (u & 1) * ACC + 32 * (half + 2 * (c >> 5)) + (c & 16);
            tmem_ld_32x32b_x16(ta, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
            if (NS == 3) {
              tmem_ld_32x32b_x16(ta + 128, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[c + j] = join(acc[c + j], v[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[u & 1]);
          ++u;
        }
      }
      if (!ok) break;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const int cc = 32 * (half + 2 * c), n = t.n0 + cc;
        if (cc >= a.s.bn || n >= g.N || mw >= g.M) break;
        Extra x;
        f2 cs[4];
        constexpr bool UA = sizeof(T) == 4 && !LONGK;
        if (EXTRA) load_extra<UA>(x, g, a.s.vec, rw, n, lane);
        epi_chunk<EPI, 16, UA>(g, a.s.vec, t.split, rw, n, c ? bias[1] : bias[0], x, cs, false, st, sbias, lane,
                           [&](int h, float (&v)[16]) {
          if constexpr (LONGK) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = NS == 3 ? SPLIT_SCALE * acc[16 * h + j] : acc[16 * h + j];
          } else {
            const uint32_t ta = tq + (u & 1) * ACC + cc + 16 * h;
            tmem_ld_32x32b_x16(ta, v);
            if (NS == 3) {
              float w[16];
              tmem_ld_32x32b_x16(ta + 128, w);
              float z = 0.f;   // 0 * v is NaN for infinities and NaN
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                v[j] += w[j];
                z = fmaf(0.f, v[j], z);
                v[j] *= SPLIT_SCALE;
              }
              if (__any_sync(0xffffffffu, z != z)) {   // (four at a time: 16 spill)
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  uint32_t hh[4], sm[4];
                  tmem_ld_cols<4>(ta + j, hh);
                  tmem_ld_cols<4>(ta + 128 + j, sm);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    v[j + k] = SPLIT_SCALE * join(__uint_as_float(hh[k]), __uint_as_float(sm[k]));
                }
              }
            }
          }
        });
        if constexpr (LONGK) {   // the next chunk's sums to the front: no index that depends on c
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] = acc[j + 32];
        }
      }
      if (!LONGK) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[u & 1]);
        ++u;
      }
    }
    if (!ok && lane == 0) atomicExch(a.err, E2F_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == CTRL_WARP) tmem_dealloc(tmem, 2 * ACC);
}

template <typename T, bool AMN, bool BMN, int EPI, int NA = 1>
static e2f_status launch(const Args &a, int sms, cudaStream_t s) {
  constexpr size_t smem = smem_bytes<T, NA>();
  if (long_chain(a.g)) {
    constexpr auto k = gemm_reg_kernel<T, AMN, BMN, EPI, true, NA>;
    E2F_CUDA_TRY(allow_smem<k>(smem, LAUNCH_REGS));
    E2F_LIN_LAUNCH(a.g, k, std::min(a.s.tiles, sms), NT, smem, s, a);
  } else {
    constexpr auto k = gemm_reg_kernel<T, AMN, BMN, EPI, false, NA>;
    E2F_CUDA_TRY(allow_smem<k>(smem, LAUNCH_REGS));
    E2F_LIN_LAUNCH(a.g, k, std::min(a.s.tiles, sms), NT, smem, s, a);
  }
  return E2F_OK;
}

}  // namespace reg

// A product whose operands have any stride and alignment, split into `splits`
// parts of g.kper contraction blocks (MODE_PART when there are several).
template <typename T, bool AMN, bool BMN>
e2f_status gemm_reg(const Gemm &g, int splits, int bn, int sms, cudaStream_t s) {
  using namespace reg;
  Args a{};
  a.g = g;
  if (!schedule(g, splits, bn, &a.s)) return E2F_ERR_UNSUPPORTED;
  a.err = device_error_flag();
  if (!a.err) return E2F_ERR_CUDA;
  if constexpr (!AMN && !BMN) {
    switch (epi_kind(g.e)) {
      case DZ: return launch<T, AMN, BMN, DZ>(a, sms, s);
      case RES: return launch<T, AMN, BMN, RES>(a, sms, s);
      case ACT: return launch<T, AMN, BMN, ACT>(a, sms, s);
      default: break;
    }
  }
  if constexpr (BMN && sizeof(T) == 2)   // the products of dz
    if (g.A2) return launch<T, AMN, BMN, PLAIN, 2>(a, sms, s);
  return launch<T, AMN, BMN, PLAIN>(a, sms, s);
}
template e2f_status gemm_reg<float, false, false>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_reg<float, false, true>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_reg<float, true, true>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_reg<__nv_bfloat16, false, false>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_reg<__nv_bfloat16, false, true>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_reg<__nv_bfloat16, true, true>(const Gemm &, int, int, int, cudaStream_t);

}  // namespace lin
}  // namespace e2f
