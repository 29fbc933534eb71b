// bf16 products of the linear layers with TMA-fed tensor cores: the path for
// operands whose rows start on 16-byte boundaries.
//
// A persistent CTA per SM walks output tiles of 128 x BN (BN = 128 or 256).
// Warp 0 loads 64-wide operand slices by TMA into a ring of stages (128-byte
// swizzle; rows and columns outside the matrices arrive as zeros), warp 1
// issues the MMAs into one of two accumulators in tensor memory, warps 4 on
// run the epilogue of the other one meanwhile: TMEM -> shared memory -> rows,
// so that residual, dL/dout and results move in 16-byte pieces of contiguous
// rows.
//
// The tensor core's fp32 accumulation truncates: a chain of s MMAs (16
// products each) leaves a relative error near s * 1e-8 (measured: 2.7e-6 at
// 256).  Where fp32 results hang on it, LONGK ends the chain every KCHUNK
// blocks and the epilogue warps add the pieces in registers, rounded to
// nearest.
#include <cuda.h>

#include <algorithm>

#include "linear.cuh"

namespace e2f {
namespace lin {

namespace tma {

constexpr int BM = 128, BK = 64;
constexpr int SHORTK = 8;                        // blocks of 64: up to here 16 epilogue warps
constexpr int KCHUNK = 16;                       // blocks of 64 per chain (LONGK)

// EW epilogue warps (8 or 16) behind the four of the control warpgroup; 16 take a quarter of the
// columns each and leave less room for the ring.
template <int EW> constexpr int threads() { return (4 + EW) * 32; }
template <int EW> constexpr int staging() { return EW * 32 * 32 * 4; }
template <int EW> constexpr int sbias() { return EW * 32 * 4; }
template <int EW> constexpr int ring() { return EW == 16 ? 147456 : 196608; }
template <int BN> constexpr int stage_bytes() { return (BM + BN) * BK * 2; }
template <int BN, int EW> constexpr int stages() { return ring<EW>() / stage_bytes<BN>(); }
template <int EW> constexpr size_t smem_bytes() { return ring<EW>() + staging<EW>() + sbias<EW>() + 256 + 1024; }

struct Args {
  Gemm g;
  int mt, nt, tiles, nkb;   // tiles: mt * nt * splits
  int vec;                  // 16-byte rows of out and extra, N a multiple of 8
  int *err;
};

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          tc::smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(tc::smem_addr(bar))
      : "memory");
}

// One operand slice: R rows (m or n) from r0, 64 contraction columns from k0.
// K-major: one box of R rows x 64; MN-major: boxes of 64 contraction rows x 64.
template <bool MN, int R>
__device__ __forceinline__ void load_slice(uint8_t *dst, const CUtensorMap *map, int r0, int k0, uint64_t *bar) {
  if (!MN) {
    tma_load_2d(dst, map, k0, r0, bar);
  } else {
#pragma unroll
    for (int j = 0; j < R / 64; ++j) tma_load_2d(dst + j * 8192, map, r0 + 64 * j, k0, bar);
  }
}

template <bool MN> __device__ __forceinline__ uint64_t slice_desc(uint32_t saddr, int k) {
  const uint32_t a = saddr + (MN ? k * 128 : k * 2);
  return tc::smem_desc(a, MN ? 8192 : 16, 1024) | (uint64_t)2 << 61;
}

struct Extra {   // 4 x 8 elements of residual or dL/dout: bf16 in lo, fp32 in lo and hi
  uint4 lo[4], hi[4];
};

struct Tile {
  int m0, n0, split, kb0, kb1, mi;
};
// Consecutive tiles share their rows of A (up to 16 column tiles, then the
// next row tile): a wave of CTAs reads few rows of A and one band of B.
template <int BN> __device__ __forceinline__ Tile tile_of(const Args &a, int i) {
  Tile t;
  const int per = a.mt * a.nt;
  t.split = i / per;
  int r = i - t.split * per;
  const int band = a.mt * 16, b = r / band;
  r -= b * band;
  const int w = min(16, a.nt - 16 * b);
  t.mi = r / w;
  t.m0 = t.mi * BM;
  t.n0 = (16 * b + r - t.mi * w) * BN;
  t.kb0 = t.split * a.g.kper;
  t.kb1 = min(t.kb0 + a.g.kper, a.nkb);
  return t;
}

__device__ __forceinline__ void unpack8(const uint4 &a, const uint4 &b, int type, float (&v)[8]) {
  if (type == E2F_F32) {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
    v[4] = __uint_as_float(a.z << 16); v[5] = __uint_as_float(a.z & 0xffff0000u);
    v[6] = __uint_as_float(a.w << 16); v[7] = __uint_as_float(a.w & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(void *p, int type, size_t i, const float (&v)[8]) {
  if (type == E2F_F32) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// EPI: what the epilogue does.  PLAIN: accumulators as they are, to out or to
// the partial sums; ACT: bias and activation; RES: those and the residual; DZ:
// MODE_DZ.  (One instance for all of them kept the registers of the last two
// alive in the others and spilled: 100,002 x 128 -> 512 with a bias 64 us.)
constexpr int PLAIN = 0, ACT = 1, RES = 2, DZ = 3;
template <bool AMN, bool BMN, int BN, bool LONGK, int EPI, int EW>
__global__ void __launch_bounds__(threads<EW>(), 1)
gemm_tma_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tbm,
                const __grid_constant__ Args a) {
  using namespace tc;
  constexpr int ST = stages<BN, EW>(), RING = ring<EW>(), STAGING = staging<EW>(), SBIAS = sbias<EW>(), SB = stage_bytes<BN>(), ABYTES = BM * BK * 2;
  constexpr uint32_t LIMIT = 1u << 26;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float *staging = reinterpret_cast<float *>(smem + RING);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + RING + STAGING + SBIAS), *empty = full + ST, *tfull = empty + ST,
           *tempty = tfull + 2;
  __shared__ uint32_t tslot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&tfull[i], 1); mbar_init(&tempty[i], EW); }
    mbar_fence_init();
  }
  __syncthreads();
  if (warp == 1) { tmem_alloc(&tslot, 2 * BN); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot;

  // LONGK: the register sums need more than the 168 that 384 threads are
  // launched with: 40 + 2 * 232 = 3 * 168.
  if (LONGK && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;   // the first pass over the ring finds it empty
      bool ok = true;
      for (int i = blockIdx.x; i < a.tiles && ok; i += gridDim.x) {
        const Tile t = tile_of<BN>(a, i);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          ok = mbar_wait(&empty[s], ph, LIMIT);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[s], SB);
          load_slice<AMN, BM>(smem + s * SB, &ta, t.m0, kb * BK, &full[s]);
          load_slice<BMN, BN>(smem + s * SB + ABYTES, &tbm, t.n0, kb * BK, &full[s]);
          if (++s == ST) { s = 0; ph ^= 1; }
        }
      }
      if (!ok) atomicExch(a.err, E2F_ERR_TIMEOUT);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0, u = 0;   // ring slot, accumulator units issued
      uint32_t ph = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < a.tiles && ok; i += gridDim.x) {
        const Tile t = tile_of<BN>(a, i);
        const int nb = min(BN, (a.g.N - t.n0 + 15) & ~15);
        const uint32_t id = idesc_bf16(128, nb, AMN, BMN);
        for (int kc = t.kb0; kc < t.kb1 && ok; kc += LONGK ? KCHUNK : t.kb1 - t.kb0, ++u) {
          const int ke = LONGK ? min(kc + KCHUNK, t.kb1) : t.kb1;
          const uint32_t acc = tmem + (u & 1) * BN;
          ok = mbar_wait(&tempty[u & 1], ((u >> 1) & 1) ^ 1, LIMIT);
          if (!ok) break;
          tc_fence_after();
          for (int kb = kc; kb < ke; ++kb) {
            ok = mbar_wait(&full[s], ph, LIMIT);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a0 = smem_addr(smem + s * SB), b0 = a0 + ABYTES;
#pragma unroll
            for (int k = 0; k < BK; k += 16)
              mma_bf16_ss(acc, slice_desc<AMN>(a0, k), slice_desc<BMN>(b0, k), id, kb > kc || k > 0 ? 1u : 0u);
            mma_commit(&empty[s]);
            if (++s == ST) { s = 0; ph ^= 1; }
          }
          mma_commit(&tfull[u & 1]);
        }
      }
      if (!ok) atomicExch(a.err, E2F_ERR_TIMEOUT);
    }
  } else if (warp >= 4) {
    if (LONGK) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    constexpr int BW = BN * 4 / EW;                              // columns of this warp
    const int ew = warp - 4, quarter = warp & 3, cols = (ew >> 2) * BW;   // TMEM lanes 32 quarter + ..
    const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16) + cols;
    float *st = staging + ew * 32 * 32;
    const Epi &e = a.g.e;
    float *sbias = reinterpret_cast<float *>(smem + RING + STAGING) + ew * 32;
    // results that need nothing more are rounded before they are staged
    const bool half_rows = EPI <= ACT && e.mode == MODE_OUT && e.otype == E2F_BF16;
    constexpr int NCH = BW / 32;   // 32-column chunks of this warp
    const int r8 = lane >> 2, cg = (lane & 3) * 8;
    int u = 0, bias_of = -1;
    float bias[NCH];
    bool ok = true;
    for (int i = blockIdx.x; i < a.tiles && ok; i += gridDim.x) {
      const Tile t = tile_of<BN>(a, i);
      const int nw = t.n0 + cols, mw = t.m0 + 32 * quarter;
      // this lane's rows r8 + 8 q of the tile, by offset and step
      const int rows = a.g.M - mw;
      const long long ldo = e.mode == MODE_PART ? a.g.N : e.ldo;
      const size_t ooff = (size_t)((long long)(mw + r8) * ldo), xoff = (size_t)((long long)(mw + r8) * e.lde);
      const long long ostep = 8 * ldo, xstep = 8 * e.lde;
      auto load_extra = [&](Extra &d, int c) {   // 8 rows x 4 pieces of 8 columns an instruction
        const int ng = nw + 32 * c + cg;
        if (!a.vec || !e.extra || ng >= a.g.N) return;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (8 * q + r8 < rows) {
            const size_t o = xoff + (size_t)(q * xstep) + ng;
            if (e.etype == E2F_F32) {
              const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(e.extra) + o);
              d.lo[q] = p[0];
              d.hi[q] = p[1];
            } else {
              d.lo[q] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(e.extra) + o);
            }
          }
        }
      };
      if (EPI != PLAIN && nw != bias_of) {   // a CTA's tiles mostly share their columns
        bias_of = nw;
#pragma unroll
        for (int k = 0; k < NCH; ++k)
          bias[k] = e.bias && nw + 32 * k + lane < a.g.N ? __ldg(e.bias + nw + 32 * k + lane) : 0.f;
      }
      constexpr bool EXTRA = EPI >= RES, AHEAD = EXTRA && !LONGK && EW == 8;   // registers for the next chunk's extra
      Extra x;
      if (AHEAD) load_extra(x, 0);
      float acc[LONGK ? BW : 1];
      if (LONGK) {
#pragma unroll
        for (int j = 0; j < BW; ++j) acc[j] = 0.f;
        for (int kc = t.kb0; kc < t.kb1; kc += KCHUNK, ++u) {
          ok = __all_sync(0xffffffffu, mbar_wait(&tfull[u & 1], (u >> 1) & 1, LIMIT));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < BW; c += 16) {
            float v[16];
            tmem_ld_32x32b_x16(tq + (u & 1) * BN + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[u & 1]);
        }
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[u & 1], (u >> 1) & 1, LIMIT));
        tc_fence_after();
      }
      if (!ok) break;
      // Not unrolled: the chunk's code fits the instruction cache once.
#pragma unroll 1
      for (int c = 0; c < NCH; ++c) {
        const int n = nw + 32 * c;
        if (n >= a.g.N || mw >= a.g.M) break;
        const int ng = n + cg;
        const bool more = c + 1 < NCH && n + 32 < a.g.N;
        Extra nx;
        if (EXTRA) {   // what the epilogue reads, on its way while the accumulators move
          if (!AHEAD) load_extra(x, c);
          else if (more) load_extra(nx, c + 1);
        }
        if (EPI != PLAIN) {
          float b = bias[0];
#pragma unroll
          for (int k = 1; k < NCH; ++k) b = k == c ? bias[k] : b;
          sbias[lane] = b;
          __syncwarp();
        }
        // lane = row: accumulators, bias, activation -> staging, PW columns at a
        // time (16 where the extra's registers live beside them)
        constexpr int PW = EXTRA && EW == 16 ? 16 : 32;
        uint4 *sh = reinterpret_cast<uint4 *>(st);
#pragma unroll
        for (int h = 0; h < 32 / PW; ++h) {
          float v[PW];
          if constexpr (LONGK) {
#pragma unroll
            for (int k = 0; k < NCH; ++k)
              if (k == c) {
#pragma unroll
                for (int j = 0; j < PW; ++j) v[j] = acc[32 * k + PW * h + j];
              }
          } else if constexpr (PW == 32) {
            tmem_ld_32x32b_x32(tq + (u & 1) * BN + 32 * c, v);
          } else {
            tmem_ld_32x32b_x16(tq + (u & 1) * BN + 32 * c + PW * h, v);
          }
          if (EPI != PLAIN) {
            if (e.bias) {
#pragma unroll
              for (int j = 0; j < PW / 4; ++j) {
                const float4 b4 = *reinterpret_cast<const float4 *>(sbias + PW * h + 4 * j);
                v[4 * j] += b4.x; v[4 * j + 1] += b4.y; v[4 * j + 2] += b4.z; v[4 * j + 3] += b4.w;
              }
            }
            if (EPI != DZ) {
              if (e.act == E2F_ACT_SILU) {
#pragma unroll
                for (int j = 0; j < PW; ++j) v[j] = silu(v[j]);
              } else if (e.act == E2F_ACT_GELU) {
#pragma unroll
                for (int j = 0; j < PW; ++j) v[j] = gelu(v[j]);
              }
            } else if (e.act == E2F_ACT_SILU) {
#pragma unroll
              for (int j = 0; j < PW; ++j) v[j] = silu_grad(v[j]);
            } else {
#pragma unroll
              for (int j = 0; j < PW; ++j) v[j] = gelu_grad(v[j]);
            }
          }
          if (half_rows) {   // bf16 results as they go out: half the shared-memory traffic
#pragma unroll
            for (int j = 0; j < PW / 8; ++j)
              sh[lane * 4 + ((PW / 8 * h + j) ^ ((lane >> 1) & 3))] =
                  make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                             pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
          } else {
#pragma unroll
            for (int j = 0; j < PW / 4; ++j)
              *reinterpret_cast<float4 *>(st + lane * 32 + (((PW / 4 * h + j) ^ (lane & 7)) << 2)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
        __syncwarp();
        if (half_rows) {
          __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out);
          if (a.vec) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = 8 * q + r8;
              const uint4 w = sh[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
              if (row < rows && ng < a.g.N) *reinterpret_cast<uint4 *>(out + ooff + (size_t)(q * ostep) + ng) = w;
            }
          } else if (n + lane < a.g.N) {
            const __nv_bfloat16 *s2 = reinterpret_cast<const __nv_bfloat16 *>(st);
#pragma unroll 8
            for (int r = 0; r < 32; ++r)
              if (mw + r < a.g.M)
                out[(size_t)((mw + r) * e.ldo) + n + lane] = s2[r * 32 + (((lane >> 3) ^ ((r >> 1) & 3)) << 3) + (lane & 7)];
          }
        } else {
          float *part = EPI != PLAIN || e.mode != MODE_PART ? nullptr : a.g.part + (size_t)t.split * a.g.M * a.g.N;
          if (a.vec) {
            float cs[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) cs[j] = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = 8 * q + r8;
              if (row < rows && ng < a.g.N) {
                const float4 lo = *reinterpret_cast<const float4 *>(st + row * 32 + (((cg >> 2) ^ (row & 7)) << 2));
                const float4 hi = *reinterpret_cast<const float4 *>(st + row * 32 + ((((cg >> 2) + 1) ^ (row & 7)) << 2));
                float r[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                if (part) {
                  store8(part, E2F_F32, ooff + (size_t)(q * ostep) + ng, r);
                  continue;
                }
                if (EXTRA) {
                  float y[8];
                  unpack8(x.lo[q], x.hi[q], e.etype, y);
                  if (EPI == RES) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[j] += y[j];
                  } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                      r[j] *= y[j];
                      cs[j] += r[j];
                    }
                  }
                }
                if (EPI != DZ || e.out) store8(e.out, e.otype, ooff + (size_t)(q * ostep) + ng, r);
              }
            }
            if (EPI == DZ && e.colpart) {   // column sums of the warp's 32 rows
#pragma unroll
              for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) cs[j] += __shfl_xor_sync(0xffffffffu, cs[j], o);
              }
              if (lane < 4 && ng < a.g.N) store8(e.colpart, E2F_F32, (size_t)(mw >> 5) * a.g.N + ng, cs);
            }
          } else if (n + lane < a.g.N) {   // any alignment: lane = column
            const int nl = n + lane;
            float cs = 0.f;
            for (int r0 = 0; r0 < 32 && mw + r0 < a.g.M; r0 += 8) {
              float y[8];
              if (EXTRA) {
#pragma unroll
                for (int r = 0; r < 8; ++r)
                  y[r] = mw + r0 + r < a.g.M ? load_as(e.extra, e.etype, (size_t)((mw + r0 + r) * e.lde) + nl) : 0.f;
              }
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                const int row = r0 + r, m = mw + row;
                if (m >= a.g.M) break;
                float w = st[row * 32 + ((((lane >> 2) ^ (row & 7)) << 2) | (lane & 3))];
                if (part) {
                  part[(size_t)m * a.g.N + nl] = w;
                  continue;
                }
                if (EXTRA) {
                  w = EPI == RES ? w + y[r] : w * y[r];
                  cs += w;
                }
                if (EPI != DZ || e.out) store_as(e.out, e.otype, (size_t)(m * e.ldo) + nl, w);
              }
            }
            if (EPI == DZ && e.colpart) e.colpart[(size_t)(mw >> 5) * a.g.N + nl] = cs;
          }
        }
        __syncwarp();
        if (AHEAD && more) x = nx;
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
  if (warp == 1) tmem_dealloc(tmem, 2 * BN);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// [rows][cols] bf16, row stride ld elements; boxes of box_rows x 64 columns.
static bool encode(CUtensorMap *m, const void *p, long long rows, long long cols, long long ld, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool AMN, bool BMN, int BN, bool LONGK, int EPI, int EW>
static e2f_status launch_epi(const CUtensorMap &ta, const CUtensorMap &tb, const Args &a, int sms, cudaStream_t s) {
  constexpr auto k = gemm_tma_kernel<AMN, BMN, BN, LONGK, EPI, EW>;
  E2F_CUDA_TRY(allow_smem<k>(smem_bytes<EW>()));
  E2F_LAUNCH(k, std::min(a.tiles, sms), threads<EW>(), smem_bytes<EW>(), s, ta, tb, a);
  return E2F_OK;
}

template <bool AMN, bool BMN, int BN, bool LONGK>
static e2f_status launch(const CUtensorMap &ta, const CUtensorMap &tb, const Args &a, int sms, cudaStream_t s) {
  const Epi &e = a.g.e;
  // A short contraction leaves the epilogue as the longer part of a tile.
  constexpr int W = LONGK ? 8 : 16;
  const bool wide = !LONGK && a.g.kper <= SHORTK;
#define E2F_LIN_EPI(E)                                                                \
  return wide ? launch_epi<AMN, BMN, BN, LONGK, E, W>(ta, tb, a, sms, s)              \
              : launch_epi<AMN, BMN, BN, LONGK, E, 8>(ta, tb, a, sms, s)
  if constexpr (!AMN && !BMN) {
    if (e.mode == MODE_DZ) E2F_LIN_EPI(DZ);
    if (e.mode == MODE_OUT && e.extra) E2F_LIN_EPI(RES);
    if (e.mode == MODE_OUT && (e.bias || e.act != E2F_ACT_NONE)) E2F_LIN_EPI(ACT);
  }
  E2F_LIN_EPI(PLAIN);
#undef E2F_LIN_EPI
}

}  // namespace tma

bool tma_operand(const void *p, long long ld) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 2)) & 15) == 0;
}

// A bf16 product of aligned operands, split into `splits` parts of g.kper
// contraction blocks (MODE_PART when there are several); bn = 128 or 256.
template <bool AMN, bool BMN>
e2f_status gemm_tma(const Gemm &g, int splits, int bn, int sms, cudaStream_t s) {
  using namespace tma;
  Args a{};
  a.g = g;
  a.mt = (g.M + BM - 1) / BM;
  a.nt = (g.N + bn - 1) / bn;
  a.nkb = (g.K + BK - 1) / BK;
  const long long tiles = (long long)a.mt * a.nt * splits;
  if (tiles > INT32_MAX / 2) return E2F_ERR_UNSUPPORTED;
  a.tiles = (int)tiles;
  a.err = device_error_flag();
  if (!a.err) return E2F_ERR_CUDA;
  auto rows16 = [](const void *p, long long ld, int type) {
    return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (type == E2F_F32 ? 4 : 2))) & 15) == 0;
  };
  a.vec = g.N % 8 == 0 && (g.e.mode == MODE_PART || (rows16(g.e.out, g.e.ldo, g.e.otype) && rows16(g.e.extra, g.e.lde, g.e.etype)));
  CUtensorMap ta, tb;
  const bool ok = (AMN ? encode(&ta, g.A, g.K, g.M, g.lda, 64) : encode(&ta, g.A, g.M, g.K, g.lda, BM)) &&
                  (BMN ? encode(&tb, g.B, g.K, g.N, g.ldb, 64) : encode(&tb, g.B, g.N, g.K, g.ldb, bn));
  if (!ok) {
    set_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    return E2F_ERR_CUDA;
  }
  const bool fp32 = g.e.mode == MODE_PART || (g.e.mode == MODE_OUT ? g.e.otype == E2F_F32 : g.e.colpart != nullptr);
  const bool longk = fp32 && g.kper > KCHUNK;
  if (bn == 256)
    return longk ? launch<AMN, BMN, 256, true>(ta, tb, a, sms, s) : launch<AMN, BMN, 256, false>(ta, tb, a, sms, s);
  return longk ? launch<AMN, BMN, 128, true>(ta, tb, a, sms, s) : launch<AMN, BMN, 128, false>(ta, tb, a, sms, s);
}
template e2f_status gemm_tma<false, false>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_tma<false, true>(const Gemm &, int, int, int, cudaStream_t);
template e2f_status gemm_tma<true, true>(const Gemm &, int, int, int, cudaStream_t);

}  // namespace lin
}  // namespace e2f
