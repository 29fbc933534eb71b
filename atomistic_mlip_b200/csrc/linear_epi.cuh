// Epilogue of the linear layers' persistent kernels: a warp takes 32 rows (its
// TMEM lanes) by 32 columns at a time from its accumulators to memory.  The
// lane holds a row while bias and activation are applied; the chunk then turns
// through shared memory so that residual, dL/dout and results move in 16-byte
// pieces of contiguous rows (one column a lane where alignment forbids that).
#pragma once

#include "linear.cuh"

namespace e2f {
namespace lin {

// What the epilogue does.  PLAIN: accumulators as they are, to out or to the
// partial sums; ACT: bias and activation; RES: those and the residual; DZ:
// MODE_DZ.  (One instance for all of them kept the registers of the last two
// alive in the others and spilled: 100,002 x 128 -> 512 with a bias 64 us
// against 35.)
constexpr int PLAIN = 0, ACT = 1, RES = 2, DZ = 3;

struct Sched {
  int mt, nt, tiles, nkb, bn;   // tiles: mt * nt * splits
  int vec;                      // 16-byte rows of out and extra, N a multiple of 8
};

struct Tile {
  int m0, n0, split, kb0, kb1;
};
// Consecutive tiles share their rows of A (up to 16 column tiles, then the
// next row tile): a wave of CTAs reads few rows of A and one band of B.
__device__ __forceinline__ Tile tile_of(const Gemm &g, const Sched &a, int i) {
  Tile t;
  const int per = a.mt * a.nt;
  t.split = i / per;
  int r = i - t.split * per;
  const int band = a.mt * 16, b = r / band;
  r -= b * band;
  const int w = min(16, a.nt - 16 * b), mi = r / w;
  t.m0 = mi * 128;
  t.n0 = (16 * b + r - mi * w) * a.bn;
  t.kb0 = t.split * g.kper;
  t.kb1 = min(t.kb0 + g.kper, a.nkb);
  return t;
}

struct Extra {   // 4 x 8 elements of residual or dL/dout: bf16 in lo, fp32 in lo and hi
  uint4 lo[4], hi[4];
};

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

// A warp's 32 rows of a tile; lane l handles rows l / 4 + 8 q, q = 0 .. 3, eight
// columns of each.
struct Rows {
  int m0, n;                     // first row, rows that exist
  size_t out, extra;             // offsets of row m0 + lane / 4
  long long ostep, xstep;        // eight rows on
};
__device__ __forceinline__ Rows rows_of(const Gemm &g, int m0, int lane) {
  Rows r;
  r.m0 = m0;
  r.n = g.M - m0;
  const long long ldo = g.e.mode == MODE_PART ? g.N : g.e.ldo, m = m0 + (lane >> 2);
  r.out = (size_t)(m * ldo);
  r.extra = (size_t)(m * g.e.lde);
  r.ostep = 8 * ldo;
  r.xstep = 8 * g.e.lde;
  return r;
}

// The chunk's residual or dL/dout from column n on.
__device__ __forceinline__ void load_extra(Extra &d, const Gemm &g, int vec, const Rows &rw, int n, int lane) {
  const Epi &e = g.e;
  const int ng = n + (lane & 3) * 8;
  if (!vec || ng >= g.N) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (8 * q + (lane >> 2) < rw.n) {
      const size_t o = rw.extra + (size_t)(q * rw.xstep) + ng;
      if (e.etype == E2F_F32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(e.extra) + o);
        d.lo[q] = p[0];
        d.hi[q] = p[1];
      } else {
        d.lo[q] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(e.extra) + o);
      }
    }
  }
}

// Columns n .. n + 31 of the warp's rows.  get(h, v) gives lane l the PW
// accumulators of row l from column n + PW h on; bias: that of column n + lane;
// x: the chunk's extra (load_extra); st: 4 KB, sbias: 32 floats of the warp.
template <int EPI, int PW, class Get>
__device__ __forceinline__ void epi_chunk(const Gemm &g, int vec, int split, const Rows &rw, int n, float bias,
                                          const Extra &x, float *st, float *sbias, int lane, Get get) {
  constexpr bool EXTRA = EPI >= RES;
  const Epi &e = g.e;
  // results that need nothing more are rounded before they are staged
  const bool half_rows = EPI <= ACT && e.mode == MODE_OUT && e.otype == E2F_BF16;
  const int r8 = lane >> 2, cg = (lane & 3) * 8, ng = n + cg, rows = rw.n;
  if (EPI != PLAIN) {
    sbias[lane] = bias;
    __syncwarp();
  }
  // lane = row: accumulators, bias, activation -> staging, PW columns at a time
  uint4 *sh = reinterpret_cast<uint4 *>(st);
#pragma unroll
  for (int h = 0; h < 32 / PW; ++h) {
    float v[PW];
    get(h, v);
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
    if (vec) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 8 * q + r8;
        const uint4 w = sh[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
        if (row < rows && ng < g.N) *reinterpret_cast<uint4 *>(out + rw.out + (size_t)(q * rw.ostep) + ng) = w;
      }
    } else if (n + lane < g.N) {
      const __nv_bfloat16 *s2 = reinterpret_cast<const __nv_bfloat16 *>(st);
#pragma unroll 8
      for (int r = 0; r < 32; ++r)
        if (rw.m0 + r < g.M)
          out[(size_t)((rw.m0 + r) * e.ldo) + n + lane] = s2[r * 32 + (((lane >> 3) ^ ((r >> 1) & 3)) << 3) + (lane & 7)];
    }
  } else {
    float *part = EPI != PLAIN || e.mode != MODE_PART ? nullptr : g.part + (size_t)split * g.M * g.N;
    if (vec) {
      float cs[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 8 * q + r8;
        if (row < rows && ng < g.N) {
          const float4 lo = *reinterpret_cast<const float4 *>(st + row * 32 + (((cg >> 2) ^ (row & 7)) << 2));
          const float4 hi = *reinterpret_cast<const float4 *>(st + row * 32 + ((((cg >> 2) + 1) ^ (row & 7)) << 2));
          float r[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          if (part) {
            store8(part, E2F_F32, rw.out + (size_t)(q * rw.ostep) + ng, r);
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
          if (EPI != DZ || e.out) store8(e.out, e.otype, rw.out + (size_t)(q * rw.ostep) + ng, r);
        }
      }
      if (EPI == DZ && e.colpart) {   // column sums of the warp's 32 rows
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) cs[j] += __shfl_xor_sync(0xffffffffu, cs[j], o);
        }
        if (lane < 4 && ng < g.N) store8(e.colpart, E2F_F32, (size_t)(rw.m0 >> 5) * g.N + ng, cs);
      }
    } else if (n + lane < g.N) {   // any alignment: lane = column
      const int nl = n + lane;
      float cs = 0.f;
      for (int r0 = 0; r0 < 32 && rw.m0 + r0 < g.M; r0 += 8) {
        float y[8];
        if (EXTRA) {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            y[r] = rw.m0 + r0 + r < g.M ? load_as(e.extra, e.etype, (size_t)((rw.m0 + r0 + r) * e.lde) + nl) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int row = r0 + r, m = rw.m0 + row;
          if (m >= g.M) break;
          float w = st[row * 32 + ((((lane >> 2) ^ (row & 7)) << 2) | (lane & 3))];
          if (part) {
            part[(size_t)m * g.N + nl] = w;
            continue;
          }
          if (EXTRA) {
            w = EPI == RES ? w + y[r] : w * y[r];
            cs += w;
          }
          if (EPI != DZ || e.out) store_as(e.out, e.otype, (size_t)(m * e.ldo) + nl, w);
        }
      }
      if (EPI == DZ && e.colpart) e.colpart[(size_t)(rw.m0 >> 5) * g.N + nl] = cs;
    }
  }
  __syncwarp();
}

// ---- host side ------------------------------------------------------------------
inline bool rows16(const void *p, long long ld, int type) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (type == E2F_F32 ? 4 : 2))) & 15) == 0;
}
// Tiles of 128 x bn, each in `splits` parts of g.kper contraction blocks of 64.
inline bool schedule(const Gemm &g, int splits, int bn, Sched *s) {
  s->mt = (g.M + 127) / 128;
  s->nt = (g.N + bn - 1) / bn;
  s->nkb = (g.K + 63) / 64;
  s->bn = bn;
  const long long tiles = (long long)s->mt * s->nt * splits;
  if (tiles > INT32_MAX / 2) return false;
  s->tiles = (int)tiles;
  const Epi &e = g.e;
  s->vec = g.N % 8 == 0 && (e.mode == MODE_PART || ((!e.out || rows16(e.out, e.ldo, e.otype)) &&
                                                    (!e.extra || rows16(e.extra, e.lde, e.etype))));
  return true;
}
inline int epi_kind(const Epi &e) {
  return e.mode == MODE_PART                       ? PLAIN
         : e.mode == MODE_DZ                       ? DZ
         : e.extra                                 ? RES
         : e.bias || e.act != E2F_ACT_NONE         ? ACT
                                                   : PLAIN;
}
// Whether fp32 results hang on the accumulators' last bits: then a chain of MMAs
// ends after KCHUNK blocks (linear_tma.cu).
constexpr int KCHUNK = 16;
inline bool long_chain(const Gemm &g) {
  const bool fp32 = g.e.mode == MODE_PART || (g.e.mode == MODE_OUT ? g.e.otype == E2F_F32 : g.e.colpart != nullptr);
  return fp32 && g.kper > KCHUNK;
}

}  // namespace lin
}  // namespace e2f
