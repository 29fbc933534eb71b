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
//
// A may come in two terms (NA = 2: dz of the backward): a stage holds a slice of
// both, B's is loaded once and multiplied with each.
//
// Measured: 8,192 x 4,096 -> 4,096 with GELU and an fp32 residual and result 217 us
// (1,270 TFLOP/s; without any of them 174, the tensor core's limit); 100,002 x 128 ->
// 512 SiLU 38 us (3.4 TB/s; without activation 25), where the epilogue's
// instructions bound it.
#include <cuda.h>

#include <algorithm>

#include "linear_epi.cuh"

namespace e2f {
namespace lin {

bool tma_operand(const void *p, long long ld) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 2)) & 15) == 0;
}

namespace tma {

constexpr int BM = 128, BK = 64;
// Contractions of up to so many blocks of 64 get 16 epilogue warps: there the
// epilogue is the longer part of a tile (4,099 x 1,000 -> 2,050, dz in one term: 45 us
// against 63; 65,536 x 768 -> 1,024 without an extra operand: 97 against 94).
constexpr int short_k(int epi) { return epi >= RES ? 16 : 8; }

// EW epilogue warps (8 or 16) behind the four of the control warpgroup; 16 take a quarter of the
// columns each and leave less room for the ring.
template <int EW> constexpr int threads() { return (4 + EW) * 32; }
template <int EW> constexpr int staging() { return EW * 32 * 32 * 4; }
template <int EW> constexpr int sbias() { return EW * 32 * 4; }
template <int EW> constexpr int ring() { return EW == 16 ? 147456 : 196608; }
template <int BN, int NA> constexpr int stage_bytes() { return (NA * BM + BN) * BK * 2; }
template <int EW> constexpr size_t smem_bytes() { return ring<EW>() + staging<EW>() + sbias<EW>() + 256 + 1024; }

struct Args {
  Gemm g;
  Sched s;
  int grid;    // CTAs
  int bres;    // bytes of B held for the whole launch (every CTA has one column tile), or 0
  int st;      // stages of the ring behind them
  int *err;
};
constexpr int MAX_ST = 12;

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

// ---- the asynchronous epilogue (IO): bf16 results, and bf16 residual or dL/dout ----
// The chunk of 32 x 32 stays with lane = row: the extra operand arrives in shared
// memory by TMA, the lane reads its row of it, writes its row of the result over
// it, and TMA takes that out.  Against turning the chunk through shared memory
// this halves the LSU wavefronts, which bound short contractions (100,002 x 128 ->
// 512: 80 % of their peak): per chunk 32 for the accumulators, 16 in, 16 out, 8
// for the bias.  Rows of 64 bytes, 64-byte swizzle.  Of a warp's three buffers the residual's chunks
// take turns in all (two loads ahead); dz, which leaves in two terms, has its second
// one in the last and dL/dout in the others, one load ahead.
constexpr int IO_BUF = 2048;
template <int EPI, int BN> constexpr int io_bufs() { return EPI >= RES ? 3 : BN / 128; }   // (a chunk or two of a tile)
template <int EPI, int BN> constexpr int io_ring() { return EPI >= RES ? 126976 : BN == 256 ? 147456 : 180224; }
constexpr int IO_SBIAS = 16 * 64 * 4;
template <int EPI, int BN> constexpr size_t io_smem() {
  return io_ring<EPI, BN>() + 16 * io_bufs<EPI, BN>() * IO_BUF + IO_SBIAS + 256 + 16 * io_bufs<EPI, BN>() * 8 + 1024;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(map),
      "r"(x), "r"(y), "r"(tc::smem_addr(src))
      : "memory");
}
// All but the N last stores of this thread have read their source.
template <int N> __device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Column sums of 32 values a lane: lane l gets that of v[l] over the warp.
__device__ __forceinline__ float transposed_sum(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float keep = up ? v[j + o] : v[j], send = up ? v[j] : v[j + o];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

template <int BN, int EPI>
__device__ __forceinline__ bool io_epilogue(const Args &a, const CUtensorMap *to, const CUtensorMap *to2,
                                            const CUtensorMap *tx, uint8_t *bufs, float *sbiases, uint64_t *xbars,
                                            uint64_t *tfull, uint64_t *tempty, uint32_t tmem, int ew, int lane) {
  using namespace tc;
  constexpr uint32_t LIMIT = 1u << 26;
  constexpr int BW = BN / 4, NCH = BW / 32, NB = io_bufs<EPI, BN>();
  constexpr int NX = EPI == DZ ? NB - 1 : NB;   // buffers that the chunks take in turn
  constexpr bool EXTRA = EPI >= RES;
  const Epi &e = a.g.e;
  const int quarter = ew & 3, cols = (ew >> 2) * BW;
  const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16) + cols;
  uint8_t *buf = bufs + ew * NB * IO_BUF;
  float *sbias = sbiases + ew * 64;
  uint64_t *xbar = xbars + ew * NB;
  const int sw = (lane >> 1) & 3;   // swizzle of this lane's row
  // lane 0's loads of the extra operand: next tile, chunk and buffer
  Tile t = tile_of(a.g, a.s, blockIdx.x), pt = t;
  int pi = blockIdx.x, pc = 0, pb = 0;
  auto load_next = [&] {
    while (pi < a.s.tiles) {
      const int n = pt.n0 + cols + 32 * pc, m = pt.m0 + 32 * quarter;
      if (pc < NCH && n < a.g.N && m < a.g.M) {
        mbar_arrive_expect_tx(&xbar[pb], IO_BUF);
        tma_load_2d(buf + pb * IO_BUF, tx, n, m, &xbar[pb]);
        ++pc;
        if (++pb == NX) pb = 0;
        return;
      }
      pi += gridDim.x;
      pc = 0;
      if (pi < a.s.tiles) next_tile(a.g, a.s, pi, &pt);
    }
  };
  if (EXTRA && lane == 0) {
    load_next();
    if (EPI != DZ) load_next();
  }
  int u = 0, b = 0, bias_of = -1;
  uint32_t xph = 0;
  float sum[NCH];
#pragma unroll
  for (int k = 0; k < NCH; ++k) sum[k] = 0.f;
  bool ok = true;
  for (int i = blockIdx.x; i < a.s.tiles && ok; i += gridDim.x) {
    if (i != (int)blockIdx.x) next_tile(a.g, a.s, i, &t);
    const int nw = t.n0 + cols, mw = t.m0 + 32 * quarter;
    if (EPI != PLAIN && nw != bias_of) {   // a CTA's tiles mostly share their columns
      bias_of = nw;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < NCH; ++k)
        sbias[32 * k + lane] = e.bias && nw + 32 * k + lane < a.g.N ? __ldg(e.bias + nw + 32 * k + lane) : 0.f;
      __syncwarp();
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&tfull[u & 1], (u >> 1) & 1, LIMIT));
    tc_fence_after();
    int c = 0;
#pragma unroll 1
    for (; ok && c < NCH; ++c) {
      const int n = nw + 32 * c;
      if (n >= a.g.N || mw >= a.g.M) break;
      float v[32];
      tmem_ld_32x32b_x32(tq + (u & 1) * BN + 32 * c, v);
      if (EPI != PLAIN) {
        if (e.bias) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 b4 = *reinterpret_cast<const float4 *>(sbias + 32 * c + 4 * j);
            const f2 p = add2({v[4 * j], v[4 * j + 1]}, {b4.x, b4.y}), q = add2({v[4 * j + 2], v[4 * j + 3]}, {b4.z, b4.w});
            v[4 * j] = p.x; v[4 * j + 1] = p.y; v[4 * j + 2] = q.x; v[4 * j + 3] = q.y;
          }
        }
#define E2F_EACH2(F)                                  \
  _Pragma("unroll") for (int j = 0; j < 32; j += 2) { \
    const f2 p = F(f2{v[j], v[j + 1]});               \
    v[j] = p.x;                                       \
    v[j + 1] = p.y;                                   \
  }
        if (EPI != DZ) {
          if (e.act == E2F_ACT_SILU) { E2F_EACH2(silu) }
          else if (e.act == E2F_ACT_GELU) { E2F_EACH2(gelu) }
        } else if (e.act == E2F_ACT_SILU) { E2F_EACH2(silu_grad) }
        else { E2F_EACH2(gelu_grad) }
#undef E2F_EACH2
      }
      uint4 *row = reinterpret_cast<uint4 *>(buf + b * IO_BUF + lane * 64);
      if (EXTRA) {
        ok = __all_sync(0xffffffffu, mbar_wait(&xbar[b], xph, LIMIT));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = row[j ^ sw];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t x = u4w(w, k);
            const f2 y = {__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)};
            const f2 z = {v[8 * j + 2 * k], v[8 * j + 2 * k + 1]}, r = EPI == RES ? add2(z, y) : mul2(z, y);
            v[8 * j + 2 * k] = r.x;
            v[8 * j + 2 * k + 1] = r.y;
          }
        }
        // the chunk before has left its buffers: the chunk after the next (dz: the next)
        // goes there
        if (lane == 0) {
          stores_read<0>();
          load_next();
        }
        if (EPI == DZ) __syncwarp();
      } else {
        if (lane == 0) stores_read<NB - 1>();
        __syncwarp();
      }
      if (EPI == DZ) {
        uint4 *rest = reinterpret_cast<uint4 *>(buf + NX * IO_BUF + lane * 64);
        if (e.out) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 h, l;
            two_terms({v[8 * j], v[8 * j + 1]}, h.x, l.x);
            two_terms({v[8 * j + 2], v[8 * j + 3]}, h.y, l.y);
            two_terms({v[8 * j + 4], v[8 * j + 5]}, h.z, l.z);
            two_terms({v[8 * j + 6], v[8 * j + 7]}, h.w, l.w);
            row[j ^ sw] = h;
            rest[j ^ sw] = l;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(to, buf + b * IO_BUF, n, mw);
            tma_store_2d(to2, buf + NX * IO_BUF, n, mw);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          row[j ^ sw] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                   pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_2d(to, buf + b * IO_BUF, n, mw);
      }
      if (++b == NX) { b = 0; xph ^= 1; }
      if (EPI == DZ && e.colpart) {
        const float s = transposed_sum(v, lane);
        if (a.s.keep) sum[0] += s;
        else if (n + lane < a.g.N) e.colpart[(size_t)(mw >> 5) * a.g.N + n + lane] = s;
        const float s0 = sum[0];   // (the sums turn by one chunk: see below)
        if (NCH == 2) { sum[0] = sum[NCH - 1]; sum[NCH - 1] = s0; }
      }
    }
    if (EPI == DZ && NCH == 2 && c == 1) {   // once around
      const float s0 = sum[0];
      sum[0] = sum[NCH - 1];
      sum[NCH - 1] = s0;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&tempty[u & 1]);
    ++u;
  }
  if (lane == 0) stores_done();
  if (EPI == DZ && a.s.keep && e.colpart) {   // row (CTA among those of its columns, quarter)
    const int n0 = t.n0 + cols;
    float *row = e.colpart + (size_t)((int)blockIdx.x / a.s.nt * 4 + quarter) * a.g.N;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
      if (n0 + 32 * k + lane < a.g.N) row[n0 + 32 * k + lane] = sum[k];
  }
  return ok;
}

// t2: A's second term (NA = 2) or the second term of the results (IO, DZ).
template <bool AMN, bool BMN, int BN, bool LONGK, int EPI, int EW, bool IO, int NA>
__global__ void __launch_bounds__(threads<EW>(), 1)
gemm_tma_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tbm,
                const __grid_constant__ CUtensorMap to, const __grid_constant__ CUtensorMap tx,
                const __grid_constant__ CUtensorMap t2, const __grid_constant__ Args a) {
  using namespace tc;
  constexpr int RING = IO ? io_ring<EPI, BN>() : ring<EW>(), STAGING = IO ? 16 * io_bufs<EPI, BN>() * IO_BUF : staging<EW>(),
                SBIAS = IO ? IO_SBIAS : sbias<EW>();
  constexpr int ATERM = BM * BK * 2, ABYTES = NA * ATERM, BBYTES = BN * BK * 2;
  static_assert(RING / (ABYTES + BBYTES) >= 2, "");
  constexpr uint32_t LIMIT = 1u << 26;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float *staging = reinterpret_cast<float *>(smem + RING);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + RING + STAGING + SBIAS), *empty = full + MAX_ST,
           *tfull = empty + MAX_ST, *tempty = tfull + 2, *bfull = tempty + 2, *xbar = full + 32;
  // (stage counts known to the compiler where B moves with A: the issuing thread
  // is on the critical path there)
  constexpr bool BRES = EW == 16;
  const int bres = BRES ? a.bres : 0;
  const int ST = BRES ? a.st : RING / (ABYTES + BBYTES), SB = bres ? ABYTES : ABYTES + BBYTES;
  uint8_t *ringp = smem + bres;
  __shared__ uint32_t tslot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&tfull[i], 1); mbar_init(&tempty[i], EW); }
    mbar_init(bfull, 1);
    if (IO && EPI >= RES)
      for (int i = 0; i < 16 * io_bufs<EPI, BN>(); ++i) mbar_init(&xbar[i], 1);
    mbar_fence_init();
  }
  __syncthreads();
  if (warp == 1) { tmem_alloc(&tslot, 2 * BN); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot;
  after_previous();

  // LONGK: the register sums need more than the 168 that 384 threads are
  // launched with: 40 + 2 * 232 = 3 * 168.
  if (LONGK && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  if (warp == 0) {
    if (lane == 0) {
      Tile t = tile_of(a.g, a.s, blockIdx.x);
      int s = 0;
      uint32_t ph = 1;   // the first pass over the ring finds it empty
      bool ok = true;
      if (bres) {
        mbar_arrive_expect_tx(bfull, bres);
        for (int kb = 0; kb < t.kb1; ++kb) load_slice<BMN, BN>(smem + kb * BBYTES, &tbm, t.n0, kb * BK, bfull);
      }
      for (int i = blockIdx.x; i < a.s.tiles && ok; i += gridDim.x) {
        if (i != (int)blockIdx.x) next_tile(a.g, a.s, i, &t);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          ok = mbar_wait(&empty[s], ph, LIMIT);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[s], SB);
          load_slice<AMN, BM>(ringp + s * SB, &ta, t.m0, kb * BK, &full[s]);
          if (NA == 2) load_slice<AMN, BM>(ringp + s * SB + ATERM, &t2, t.m0, kb * BK, &full[s]);
          if (!bres) load_slice<BMN, BN>(ringp + s * SB + ABYTES, &tbm, t.n0, kb * BK, &full[s]);
          if (++s == ST) { s = 0; ph ^= 1; }
        }
      }
      if (!ok) atomicExch(a.err, E2F_ERR_TIMEOUT);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Tile t = tile_of(a.g, a.s, blockIdx.x);
      int s = 0, u = 0;   // ring slot, accumulator units issued
      uint32_t ph = 0;
      bool ok = !bres || mbar_wait(bfull, 0, LIMIT);
      for (int i = blockIdx.x; i < a.s.tiles && ok; i += gridDim.x) {
        if (i != (int)blockIdx.x) next_tile(a.g, a.s, i, &t);
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
            const uint32_t a0 = smem_addr(ringp + s * SB), b0 = bres ? smem_addr(smem + kb * BBYTES) : a0 + ABYTES;
#pragma unroll
            for (int k = 0; k < BK; k += 16) {
              mma_bf16_ss(acc, slice_desc<AMN>(a0, k), slice_desc<BMN>(b0, k), id, kb > kc || k > 0 ? 1u : 0u);
              if (NA == 2) mma_bf16_ss(acc, slice_desc<AMN>(a0 + ATERM, k), slice_desc<BMN>(b0, k), id, 1u);
            }
            mma_commit(&empty[s]);
            if (++s == ST) { s = 0; ph ^= 1; }
          }
          mma_commit(&tfull[u & 1]);
        }
      }
      if (!ok) atomicExch(a.err, E2F_ERR_TIMEOUT);
    }
  } else if (IO && warp >= 4) {
    const bool ok = io_epilogue<BN, EPI>(a, &to, &t2, &tx, smem + RING, reinterpret_cast<float *>(smem + RING + STAGING), xbar,
                                         tfull, tempty, tmem, warp - 4, lane);
    if (!ok && lane == 0) atomicExch(a.err, E2F_ERR_TIMEOUT);
  } else if (!IO && warp >= 4) {
    if (LONGK) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    constexpr int BW = BN * 4 / EW;                              // columns of this warp
    const int ew = warp - 4, quarter = warp & 3, cols = (ew >> 2) * BW;   // TMEM lanes 32 quarter + ..
    const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16) + cols;
    float *st = staging + ew * 32 * 32;
    const Epi &e = a.g.e;
    float *sbias = reinterpret_cast<float *>(smem + RING + STAGING) + ew * 32;
    constexpr int NCH = BW / 32;   // 32-column chunks of this warp
    int u = 0, bias_of = -1;
    float bias[NCH];
    f2 sums[EPI == DZ ? NCH : 1][4];
    if (EPI == DZ) {
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[k][j] = both(0.f);
    }
    bool ok = true;
    Tile t = tile_of(a.g, a.s, blockIdx.x);
    for (int i = blockIdx.x; i < a.s.tiles && ok; i += gridDim.x) {
      if (i != (int)blockIdx.x) next_tile(a.g, a.s, i, &t);
      const int nw = t.n0 + cols, mw = t.m0 + 32 * quarter;
      const Rows rw = rows_of(a.g, t.split, mw, lane);
      if (EPI != PLAIN && nw != bias_of) {   // a CTA's tiles mostly share their columns
        bias_of = nw;
#pragma unroll
        for (int k = 0; k < NCH; ++k)
          bias[k] = e.bias && nw + 32 * k + lane < a.g.N ? __ldg(e.bias + nw + 32 * k + lane) : 0.f;
      }
      constexpr bool EXTRA = EPI >= RES, AHEAD = EXTRA && !LONGK && EW == 8;   // registers for the next chunk's extra
      Extra x;
      if (AHEAD && nw < a.g.N && mw < a.g.M) load_extra<false>(x, a.g, a.s.vec, rw, nw, lane);
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
      // Not unrolled: the chunk's code fits the instruction cache once.  What a
      // chunk keeps in registers is always at the front of its array, which
      // turns by one chunk each time: an index that depends on c would put the
      // arrays into memory.
      auto turn = [&] {
        const float b0 = bias[0];
#pragma unroll
        for (int k = 0; k + 1 < NCH; ++k) bias[k] = bias[k + 1];
        bias[NCH - 1] = b0;
        if constexpr (EPI == DZ) {
          f2 s0[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) s0[j] = sums[0][j];
#pragma unroll
          for (int k = 0; k + 1 < NCH; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[k][j] = sums[k + 1][j];
#pragma unroll
          for (int j = 0; j < 4; ++j) sums[NCH - 1][j] = s0[j];
        }
      };
      int c = 0;
#pragma unroll 1
      for (; c < NCH; ++c) {
        const int n = nw + 32 * c;
        if (n >= a.g.N || mw >= a.g.M) break;
        const bool more = c + 1 < NCH && n + 32 < a.g.N;
        Extra nx;
        if (EXTRA) {   // what the epilogue reads, on its way while the accumulators move
          if (!AHEAD) load_extra<false>(x, a.g, a.s.vec, rw, n, lane);
          else if (more) load_extra<false>(nx, a.g, a.s.vec, rw, n + 32, lane);
        }
        // (16 columns at a time where the extra's registers live beside them)
        constexpr int PW = EXTRA && EW == 16 ? 16 : 32;
        epi_chunk<EPI, PW, false>(a.g, a.s.vec, t.split, rw, n, bias[0], x, sums[0], a.s.keep, st, sbias, lane,
                           [&](int h, float (&v)[PW]) {
          if constexpr (LONGK) {
#pragma unroll
            for (int j = 0; j < PW; ++j) v[j] = acc[PW * h + j];
          } else if constexpr (PW == 32) {
            tmem_ld_32x32b_x32(tq + (u & 1) * BN + 32 * c, v);
          } else {
            tmem_ld_32x32b_x16(tq + (u & 1) * BN + 32 * c + PW * h, v);
          }
        });
        if (AHEAD && more) x = nx;
        turn();
        if constexpr (LONGK) {
#pragma unroll
          for (int j = 0; j + 32 < BW; ++j) acc[j] = acc[j + 32];
        }
      }
      for (; c < NCH; ++c) turn();   // once around
      if (!LONGK) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[u & 1]);
        ++u;
      }
    }
    if (EPI == DZ && a.s.keep && e.colpart) {   // row (CTA among those of its columns, quarter)
      const int n0 = t.n0 + cols;
      float *row = a.g.e.colpart + (size_t)((int)blockIdx.x / a.s.nt * 4 + quarter) * a.g.N;
#pragma unroll
      for (int k = 0; k < NCH; ++k)
        if (n0 + 32 * k < a.g.N) flush_colsum(sums[k], row, n0 + 32 * k + (lane & 3) * 8, a.g.N, lane);
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

// [rows][cols] bf16, row stride ld elements; boxes of box_rows x box_cols (64:
// 128-byte swizzle, 32: 64-byte).
static bool encode(CUtensorMap *m, const void *p, long long rows, long long cols, long long ld, int box_rows,
                   int box_cols = 64) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool AMN, bool BMN, int BN, bool LONGK, int EPI, int EW, bool IO, int NA>
static e2f_status launch_epi(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &ta2, Args a, cudaStream_t s) {
  // B stays in shared memory for the launch where every CTA has one column tile
  // and five stages of A fit beside it (with three, too few bytes in flight:
  // 100,002 x 512 -> 128 33 us, 30 with B in the ring).
  constexpr int RING = IO ? io_ring<EPI, BN>() : ring<EW>();
  const long long bres = (long long)a.s.nkb * BN * BK * 2, abytes = NA * BM * BK * 2;
  a.bres = EW == 16 && a.s.fixed && a.g.kper == a.s.nkb && bres + 5 * abytes <= RING ? (int)bres : 0;
  a.st = std::min<int>(MAX_ST, (RING - a.bres) / (a.bres ? (int)abytes : stage_bytes<BN, NA>()));
  CUtensorMap to{}, tx{}, t2 = ta2;
  if (IO) {
    const Epi &e = a.g.e;
    if ((e.out && !encode(&to, e.out, a.g.M, a.g.N, e.ldo, 32, 32)) ||
        (EPI == DZ && e.out2 && !encode(&t2, e.out2, a.g.M, a.g.N, e.ldo, 32, 32)) ||
        (EPI >= RES && !encode(&tx, e.extra, a.g.M, a.g.N, e.lde, 32, 32))) {
      set_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
      return E2F_ERR_CUDA;
    }
  }
  constexpr auto k = gemm_tma_kernel<AMN, BMN, BN, LONGK, EPI, EW, IO, NA>;
  constexpr size_t smem = IO ? io_smem<EPI, BN>() : smem_bytes<EW>();
  E2F_CUDA_TRY(allow_smem<k>(smem, LONGK ? 168 : 0));
  E2F_LIN_LAUNCH(a.g, k, a.grid, threads<EW>(), smem, s, ta, tb, to, tx, t2, a);
  return E2F_OK;
}

template <bool AMN, bool BMN, int BN, bool LONGK, int EPI, int NA>
static e2f_status launch_kind(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &ta2, const Args &a, cudaStream_t s) {
  if constexpr (!LONGK) {
    const Epi &e = a.g.e;
    if (a.g.kper <= short_k(EPI)) {
      // (a dz that is not stored takes the same kernel: its column sums have one order)
      const bool io = e.mode != MODE_PART && e.otype == E2F_BF16 && (e.out ? tma_operand(e.out, e.ldo) : EPI == DZ) &&
                      (EPI < RES || (e.etype == E2F_BF16 && tma_operand(e.extra, e.lde)));
      if (io) return launch_epi<AMN, BMN, BN, false, EPI, 16, true, NA>(ta, tb, ta2, a, s);
      return launch_epi<AMN, BMN, BN, false, EPI, 16, false, NA>(ta, tb, ta2, a, s);
    }
  }
  return launch_epi<AMN, BMN, BN, LONGK, EPI, 8, false, NA>(ta, tb, ta2, a, s);
}

template <bool AMN, bool BMN, int BN, bool LONGK>
static e2f_status launch(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &ta2, const Args &a, cudaStream_t s) {
  if constexpr (!AMN && !BMN) {
    switch (epi_kind(a.g.e)) {
      case DZ: return launch_kind<AMN, BMN, BN, LONGK, DZ, 1>(ta, tb, ta2, a, s);
      case RES: return launch_kind<AMN, BMN, BN, LONGK, RES, 1>(ta, tb, ta2, a, s);
      case ACT: return launch_kind<AMN, BMN, BN, LONGK, ACT, 1>(ta, tb, ta2, a, s);
      default: break;
    }
  }
  if constexpr (BMN)   // the products of dz
    if (a.g.A2) return launch_kind<AMN, BMN, BN, LONGK, PLAIN, 2>(ta, tb, ta2, a, s);
  return launch_kind<AMN, BMN, BN, LONGK, PLAIN, 1>(ta, tb, ta2, a, s);
}

}  // namespace tma

// A bf16 product of aligned operands, split into `splits` parts of g.kper
// contraction blocks (MODE_PART when there are several); bn = 128 or 256.
template <bool AMN, bool BMN>
e2f_status gemm_tma(const Gemm &g, int splits, int bn, int sms, cudaStream_t s, int *rows_out) {
  using namespace tma;
  Args a{};
  a.g = g;
  if (!schedule(g, splits, bn, &a.s)) return E2F_ERR_UNSUPPORTED;
  a.err = device_error_flag();
  if (!a.err) return E2F_ERR_CUDA;
  // A grid that is a multiple of the column tiles gives each CTA one of them
  // (where that takes no further wave of tiles).
  a.grid = std::min(a.s.tiles, sms);
  const int even = a.s.nt <= 16 && splits == 1 ? a.grid / a.s.nt * a.s.nt : 0;
  if (even > 0 && (a.s.tiles + even - 1) / even == (a.s.tiles + a.grid - 1) / a.grid) {
    a.grid = even;
    a.s.fixed = 1;
    a.s.dm = even / a.s.nt * 128;
    if (g.e.mode == MODE_DZ && a.s.vec) {
      a.s.keep = 1;
      if (rows_out) *rows_out = even / a.s.nt * 4;
    }
  }
  CUtensorMap ta, tb, ta2{};
  auto encode_a = [&](CUtensorMap *m, const void *p) {
    return AMN ? encode(m, p, g.K, g.M, g.lda, 64) : encode(m, p, g.M, g.K, g.lda, BM);
  };
  const bool ok = encode_a(&ta, g.A) && (!g.A2 || encode_a(&ta2, g.A2)) &&
                  (BMN ? encode(&tb, g.B, g.K, g.N, g.ldb, 64) : encode(&tb, g.B, g.N, g.K, g.ldb, bn));
  if (!ok) {
    set_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    return E2F_ERR_CUDA;
  }
  const bool longk = long_chain(g);
  if (bn == 256)
    return longk ? launch<AMN, BMN, 256, true>(ta, tb, ta2, a, s) : launch<AMN, BMN, 256, false>(ta, tb, ta2, a, s);
  return longk ? launch<AMN, BMN, 128, true>(ta, tb, ta2, a, s) : launch<AMN, BMN, 128, false>(ta, tb, ta2, a, s);
}
template e2f_status gemm_tma<false, false>(const Gemm &, int, int, int, cudaStream_t, int *);
template e2f_status gemm_tma<false, true>(const Gemm &, int, int, int, cudaStream_t, int *);
template e2f_status gemm_tma<true, true>(const Gemm &, int, int, int, cudaStream_t, int *);

}  // namespace lin
}  // namespace e2f
