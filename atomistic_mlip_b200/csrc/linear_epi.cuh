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
  int fixed;                    // a CTA's tiles share their columns ...
  int dm;                       // ... and are so many rows apart
  int keep;                     // DZ: ... whose sums stay in registers
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
// The CTA's tile i behind the one before (tile_of's divisions were a fifth of a
// short contraction's epilogue).
__device__ __forceinline__ void next_tile(const Gemm &g, const Sched &a, int i, Tile *t) {
  if (a.fixed) t->m0 += a.dm;
  else *t = tile_of(g, a, i);
}

// A chunk's residual or dL/dout: 4 x 8 elements, bf16 in lo, fp32 in lo and hi;
// where rows are not aligned, column n + lane of the 32 rows, a word each.
struct Extra {
  uint4 lo[4], hi[4];
  __device__ __forceinline__ uint32_t word(int r) const { return r < 16 ? u4w(lo[r >> 2], r & 3) : u4w(hi[(r - 16) >> 2], r & 3); }
  __device__ __forceinline__ void word(int r, uint32_t v) {
    uint4 &q = r < 16 ? lo[r >> 2] : hi[(r - 16) >> 2];
    if ((r & 3) == 0) q.x = v;
    else if ((r & 3) == 1) q.y = v;
    else if ((r & 3) == 2) q.z = v;
    else q.w = v;
  }
};

// Eight elements of type T (float, __nv_bfloat16) as four pairs, from the raw words.
template <typename T> __device__ __forceinline__ void unpack8(const uint4 &a, const uint4 &b, f2 (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = {__uint_as_float(a.x), __uint_as_float(a.y)};
    v[1] = {__uint_as_float(a.z), __uint_as_float(a.w)};
    v[2] = {__uint_as_float(b.x), __uint_as_float(b.y)};
    v[3] = {__uint_as_float(b.z), __uint_as_float(b.w)};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = u4w(a, i);
      v[i] = {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
    }
  }
}
template <typename T> __device__ __forceinline__ void store8(char *p, const f2 (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                               pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
  }
}

// A warp's 32 rows of a tile; lane l handles rows l / 4 + 8 q, q = 0 .. 3, eight
// columns of each.  Addresses in bytes.
struct Rows {
  int m0, n;                     // first row, rows that exist
  char *out;                     // row m0 + lane / 4 of the results (or partial sums)
  const char *extra;
  long long ostep, xstep;        // eight rows on
  long long rest;                // from out to out2, 0 if there is none
};
__device__ __forceinline__ Rows rows_of(const Gemm &g, int split, int m0, int lane) {
  Rows r;
  r.m0 = m0;
  r.n = g.M - m0;
  const long long m = m0 + (lane >> 2);
  if (g.e.mode == MODE_PART) {
    r.out = reinterpret_cast<char *>(g.part) + (((size_t)split * g.M + m) * g.N) * 4;
    r.ostep = 32LL * g.N;
  } else {
    const int sz = g.e.otype == E2F_F32 ? 4 : 2;
    r.out = static_cast<char *>(g.e.out) + (size_t)(m * g.e.ldo) * sz;
    r.ostep = 8 * g.e.ldo * sz;
  }
  r.rest = g.e.out2 ? static_cast<char *>(g.e.out2) - static_cast<char *>(g.e.out) : 0;
  const int xz = g.e.etype == E2F_F32 ? 4 : 2;
  r.extra = static_cast<const char *>(g.e.extra) + (size_t)(m * g.e.lde) * xz;
  r.xstep = 8 * g.e.lde * xz;
  return r;
}

// The chunk's residual or dL/dout from column n on; UA: rows of any alignment too.
template <bool UA>
__device__ __forceinline__ void load_extra(Extra &d, const Gemm &g, int vec, const Rows &rw, int n, int lane) {
  const int ng = n + (lane & 3) * 8, r8 = lane >> 2;
  if (!vec) {
    if (!UA || n + lane >= g.N) return;
    if (g.e.etype == E2F_F32) {
      const uint32_t *p = static_cast<const uint32_t *>(g.e.extra) + (size_t)(rw.m0 * g.e.lde) + n + lane;
#pragma unroll
      for (int r = 0; r < 32; ++r, p += g.e.lde)
        if (r < rw.n) d.word(r, __ldg(p));
    } else {
      const unsigned short *p = static_cast<const unsigned short *>(g.e.extra) + (size_t)(rw.m0 * g.e.lde) + n + lane;
#pragma unroll
      for (int r = 0; r < 32; ++r, p += g.e.lde)
        if (r < rw.n) d.word(r, (uint32_t)__ldg(p) << 16);
    }
    return;
  }
  if (ng >= g.N) return;
  if (g.e.etype == E2F_F32) {
    const char *p = rw.extra + 4 * (size_t)ng;
#pragma unroll
    for (int q = 0; q < 4; ++q, p += rw.xstep)
      if (8 * q + r8 < rw.n) {
        d.lo[q] = reinterpret_cast<const uint4 *>(p)[0];
        d.hi[q] = reinterpret_cast<const uint4 *>(p)[1];
      }
  } else {
    const char *p = rw.extra + 2 * (size_t)ng;
#pragma unroll
    for (int q = 0; q < 4; ++q, p += rw.xstep)
      if (8 * q + r8 < rw.n) d.lo[q] = *reinterpret_cast<const uint4 *>(p);
  }
}

// Column sums over a warp's rows: lane's eight columns of a chunk -> all rows
// (lanes 4 apart hold the same columns), lanes 0 .. 3 write.
__device__ __forceinline__ void flush_colsum(f2 (&cs)[4], float *row, int ng, int N, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
      cs[j] = add2(cs[j], {__shfl_xor_sync(0xffffffffu, cs[j].x, o), __shfl_xor_sync(0xffffffffu, cs[j].y, o)});
  }
  if (lane < 4 && ng < N) store8<float>(reinterpret_cast<char *>(row + ng), cs);
}

// Rows of a chunk from fp32 staging to memory, with the residual or dL/dout.
template <int EPI, typename XT, typename OT>
__device__ __forceinline__ void put_rows(const Rows &rw, const Extra &x, const float *st, f2 (&cs)[4], bool store, int ng,
                                         int N, int lane) {
  const int r8 = lane >> 2, c4 = (lane & 3) * 2;
  char *o = rw.out + sizeof(OT) * (size_t)ng;
#pragma unroll
  for (int q = 0; q < 4; ++q, o += rw.ostep) {
    const int row = 8 * q + r8;
    if (row >= rw.n || ng >= N) continue;
    const float4 lo = *reinterpret_cast<const float4 *>(st + row * 32 + ((c4 ^ (row & 7)) << 2));
    const float4 hi = *reinterpret_cast<const float4 *>(st + row * 32 + (((c4 + 1) ^ (row & 7)) << 2));
    f2 r[4] = {{lo.x, lo.y}, {lo.z, lo.w}, {hi.x, hi.y}, {hi.z, hi.w}};
    if constexpr (EPI >= RES) {
      f2 y[4];
      unpack8<XT>(x.lo[q], x.hi[q], y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = EPI == RES ? add2(r[j], y[j]) : mul2(r[j], y[j]);
        if (EPI == DZ) cs[j] = add2(cs[j], r[j]);
      }
    }
    if (EPI == DZ && sizeof(OT) == 2) {
      if (store) {
        uint4 h, l;
        two_terms(r[0], h.x, l.x);
        two_terms(r[1], h.y, l.y);
        two_terms(r[2], h.z, l.z);
        two_terms(r[3], h.w, l.w);
        *reinterpret_cast<uint4 *>(o) = h;
        *reinterpret_cast<uint4 *>(o + rw.rest) = l;
      }
    } else if (store) {
      store8<OT>(o, r);
    }
  }
}

// Columns n .. n + 31 of the warp's rows.  get(h, v) gives lane l the PW
// accumulators of row l from column n + PW h on; bias: that of column n + lane;
// x: the chunk's extra (load_extra); st: 4 KB, sbias: 32 floats of the warp.
// DZ: the lane's column sums are added to cs where that is kept across tiles
// (keep), else go to their row of e.colpart.
// UA: an unaligned chunk's extra was loaded with it and its 32 rows are unrolled.
// Only the fp32 kernel does: 80,736 x 79 -> 429 172 -> 137 us there, while the
// registers that it takes cost the others more (bf16 75 -> 86 us; aligned fp32
// residuals of 8,192 x 1,024 -> 4,096 83 -> 90 us).
template <int EPI, int PW, bool UA, class Get>
__device__ __forceinline__ void epi_chunk(const Gemm &g, int vec, int split, const Rows &rw, int n, float bias,
                                          const Extra &x, f2 (&cs)[4], bool keep, float *st, float *sbias, int lane,
                                          Get get) {
  constexpr bool EXTRA = EPI >= RES;
  const Epi &e = g.e;
  // results that need nothing more are rounded before they are staged
  const bool half_rows = EPI <= ACT && e.mode == MODE_OUT && e.otype == E2F_BF16;
  const int r8 = lane >> 2, ng = n + (lane & 3) * 8;
  if (EPI != PLAIN) {
    sbias[lane] = bias;
    __syncwarp();
  }
  // lane = row: accumulators, bias, activation -> staging, PW columns at a time
  uint4 *sh = reinterpret_cast<uint4 *>(st);
#pragma unroll
  for (int h = 0; h < 32 / PW; ++h) {
    f2 v[PW / 2];
    {
      float w[PW];
      get(h, w);
#pragma unroll
      for (int j = 0; j < PW / 2; ++j) v[j] = {w[2 * j], w[2 * j + 1]};
    }
    if (EPI != PLAIN) {
      if (e.bias) {
#pragma unroll
        for (int j = 0; j < PW / 4; ++j) {
          const float4 b4 = *reinterpret_cast<const float4 *>(sbias + PW * h + 4 * j);
          v[2 * j] = add2(v[2 * j], {b4.x, b4.y});
          v[2 * j + 1] = add2(v[2 * j + 1], {b4.z, b4.w});
        }
      }
      if (EPI != DZ) {
        if (e.act == E2F_ACT_SILU) {
#pragma unroll
          for (int j = 0; j < PW / 2; ++j) v[j] = silu(v[j]);
        } else if (e.act == E2F_ACT_GELU) {
#pragma unroll
          for (int j = 0; j < PW / 2; ++j) v[j] = gelu(v[j]);
        }
      } else if (e.act == E2F_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < PW / 2; ++j) v[j] = silu_grad(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < PW / 2; ++j) v[j] = gelu_grad(v[j]);
      }
    }
    if (half_rows) {   // bf16 results as they go out: half the shared-memory traffic
#pragma unroll
      for (int j = 0; j < PW / 8; ++j)
        sh[lane * 4 + ((PW / 8 * h + j) ^ ((lane >> 1) & 3))] =
            make_uint4(pack_bf16x2(v[4 * j].x, v[4 * j].y), pack_bf16x2(v[4 * j + 1].x, v[4 * j + 1].y),
                       pack_bf16x2(v[4 * j + 2].x, v[4 * j + 2].y), pack_bf16x2(v[4 * j + 3].x, v[4 * j + 3].y));
    } else {
#pragma unroll
      for (int j = 0; j < PW / 4; ++j)
        *reinterpret_cast<float4 *>(st + lane * 32 + (((PW / 4 * h + j) ^ (lane & 7)) << 2)) =
            make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
    }
  }
  __syncwarp();
  if (half_rows) {
    if (vec) {
      char *o = rw.out + 2 * (size_t)ng;
#pragma unroll
      for (int q = 0; q < 4; ++q, o += rw.ostep) {
        const int row = 8 * q + r8;
        const uint4 w = sh[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
        if (row < rw.n && ng < g.N) *reinterpret_cast<uint4 *>(o) = w;
      }
    } else if (n + lane < g.N) {
      const __nv_bfloat16 *s2 = reinterpret_cast<const __nv_bfloat16 *>(st);
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out) + (size_t)(rw.m0 * e.ldo) + n + lane;
#pragma unroll 8
      for (int r = 0; r < 32; ++r, out += e.ldo)
        if (r < rw.n) *out = s2[r * 32 + (((lane >> 3) ^ ((r >> 1) & 3)) << 3) + (lane & 7)];
    }
  } else if (vec) {
    if (EPI == DZ && !keep) {
#pragma unroll
      for (int j = 0; j < 4; ++j) cs[j] = both(0.f);
    }
    const bool store = EPI != DZ || e.out, xf = e.etype == E2F_F32, of = e.mode == MODE_PART || e.otype == E2F_F32;
    if constexpr (EPI == DZ) {
      if (xf && of) put_rows<EPI, float, float>(rw, x, st, cs, store, ng, g.N, lane);
      else if (xf) put_rows<EPI, float, __nv_bfloat16>(rw, x, st, cs, store, ng, g.N, lane);
      else if (of) put_rows<EPI, __nv_bfloat16, float>(rw, x, st, cs, store, ng, g.N, lane);
      else put_rows<EPI, __nv_bfloat16, __nv_bfloat16>(rw, x, st, cs, store, ng, g.N, lane);
    } else {   // the residual has the results' type
      if (of) put_rows<EPI, float, float>(rw, x, st, cs, store, ng, g.N, lane);
      else put_rows<EPI, __nv_bfloat16, __nv_bfloat16>(rw, x, st, cs, store, ng, g.N, lane);
    }
    if (EPI == DZ && !keep && e.colpart) flush_colsum(cs, e.colpart + (size_t)(rw.m0 >> 5) * g.N, ng, g.N, lane);
  } else if (n + lane < g.N) {   // any alignment: lane = column
    const int nl = n + lane;
    float sum = 0.f;
    if constexpr (UA) {
      const bool of = e.mode == MODE_PART || e.otype == E2F_F32, store = EPI != DZ || e.out;
      char *o = rw.out - (size_t)((long long)r8 * (rw.ostep / 8)) + (of ? 4 : 2) * (size_t)nl;   // row m0
#pragma unroll
      for (int r = 0; r < 32; ++r, o += rw.ostep / 8) {
        if (r < rw.n) {
          float w = st[r * 32 + ((((lane >> 2) ^ (r & 7)) << 2) | (lane & 3))];
          if (EXTRA) {
            const float y = __uint_as_float(x.word(r));
            w = EPI == RES ? w + y : __fmul_rn(w, y);
            sum += w;
          }
          if (store) {   // (UA: fp32 operands, so without a second term)
            if (of) *reinterpret_cast<float *>(o) = w;
            else *reinterpret_cast<__nv_bfloat16 *>(o) = __float2bfloat16_rn(w);
          }
        }
      }
    } else {
      float *part = EPI != PLAIN || e.mode != MODE_PART ? nullptr : g.part + (size_t)split * g.M * g.N;
      for (int r0 = 0; r0 < 32 && r0 < rw.n; r0 += 8) {
        float y[8];
        if (EXTRA) {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            y[r] = r0 + r < rw.n ? load_as(e.extra, e.etype, (size_t)((rw.m0 + r0 + r) * e.lde) + nl) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int row = r0 + r, m = rw.m0 + row;
          if (row >= rw.n) break;
          float w = st[row * 32 + ((((lane >> 2) ^ (row & 7)) << 2) | (lane & 3))];
          if (part) {
            part[(size_t)m * g.N + nl] = w;
            continue;
          }
          if (EXTRA) {
            w = EPI == RES ? w + y[r] : __fmul_rn(w, y[r]);
            sum += w;
          }
          const size_t i = (size_t)(m * e.ldo) + nl;
          if (EPI == DZ && e.out2) {
            two_terms(w, static_cast<__nv_bfloat16 *>(e.out)[i], static_cast<__nv_bfloat16 *>(e.out2)[i]);
          } else if (EPI != DZ || e.out) {
            store_as(e.out, e.otype, i, w);
          }
        }
      }
    }
    if (EPI == DZ && e.colpart) e.colpart[(size_t)(rw.m0 >> 5) * g.N + nl] = sum;
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
  // (dz whether its column sums are asked for or not: any subset of the gradients has
  // the bits of all of them)
  const bool fp32 = g.e.mode != MODE_OUT || g.e.otype == E2F_F32;
  return fp32 && g.kper > KCHUNK;
}

}  // namespace lin
}  // namespace e2f
