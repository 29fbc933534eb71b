// How the embedding gradient divides its rows: tiles of the sort and of the run
// sums, passes, the warp's search in the sorted keys.  Plain arithmetic, host and
// device; every count and index fits 32 bits for up to 2^31 - 4096 rows and ids,
// but sums of them need not, so those are formed in 64.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define E2F_PLAN __host__ __device__ __forceinline__
#else
#define E2F_PLAN inline
#endif

namespace e2f {
namespace emb {

constexpr int SUB = 2048;        // keys a CTA of the sort ranks at a time: 8 warps x 256
constexpr int MAX_TILES = 128;   // CTAs of a sort pass; longer inputs give each more keys
constexpr int ZROWS = 64;        // ids a CTA looks at for those that do not occur
constexpr int RED_NT = 256;      // threads of a run-sum CTA
constexpr int RED_CTAS = 4;      // ... of which so many are resident

struct SortPlan {
  int tile, tiles;   // keys of a CTA, a multiple of SUB; CTAs
  int passes;        // of 8 bits: keys run over 0 .. V (V: rows that take no part)
};
E2F_PLAN SortPlan sort_plan(int64_t N, int64_t V) {
  SortPlan p;
  const int64_t subs = (N + SUB - 1) / SUB, per = (subs + MAX_TILES - 1) / MAX_TILES, tile = per * SUB;
  p.tile = (int)tile;
  p.tiles = (int)((N + tile - 1) / tile);
  p.passes = 1;
  while (8 * p.passes < 32 && (V >> (8 * p.passes)) != 0) ++p.passes;
  return p;
}

struct RunPlan {
  int CL;        // lanes over the columns
  int R, tiles;  // places of a CTA; tiles of the sorted order
  int zero;      // CTAs that look for ids that do not occur
};
// dv: vectors of a row.
E2F_PLAN RunPlan run_plan(int64_t N, int64_t V, int dv) {
  RunPlan p;
  p.CL = 8;   // eight lanes at least: the row groups are joined one after another
  while (p.CL < 32 && p.CL < dv) p.CL <<= 1;
  // rows of a group: a multiple of eight (batches of loads) that lets one wave
  // of CTAs cover everything, 32 at most (100,002 rows, D = 128: 24 rows 12 us,
  // 16 rows, a wave and a bit, 18 us)
  const int64_t RG = RED_NT / p.CL, cols = ((int64_t)dv + p.CL - 1) / p.CL, slots = 148 * RED_CTAS;
  int64_t G = 8 * (((N + 8 * RG - 1) / (8 * RG) * cols + slots - 1) / slots);
  if (G > 32) G = 32;
  p.R = (int)(RG * G < 1024 ? RG * G : 1024);
  p.tiles = (int)((N + p.R - 1) / p.R);
  p.zero = (int)((V + ZROWS - 1) / ZROWS);
  return p;
}

// A step of the search for the first of n sorted keys >= v, by 32 lanes: the bound
// is in [lo, hi], keys[lo - 1] < v <= keys[hi].  Probes at or behind hi count as
// keys >= v; f is the first such probe, 32 if there is none.
E2F_PLAN int probe_step(int lo, int hi) { return (hi - lo + 31) >> 5; }
E2F_PLAN int probe_at(int lo, int step, int lane) { return lo + (lane + 1) * step - 1; }
E2F_PLAN void narrow(int &lo, int &hi, int step, int f) {
  if (f < 32) {
    const int p = probe_at(lo, step, f);
    if (p < hi) hi = p;
  }
  lo += f * step;
  if (lo > hi) lo = hi;
}

}  // namespace emb
}  // namespace e2f
