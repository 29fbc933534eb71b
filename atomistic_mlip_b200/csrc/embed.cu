// Scaled embedding lookup (ids -> the l = 0 rows of node features) and its
// gradient by sorted ids.
//
//   out[n][0][:] = scale * table[id_n],  out[n][q > 0][:] = 0
//   grad_table[v][:] = scale * sum over {n : id_n = v} of grad_out[n][0][:]
//
// Both are bound by HBM: the lookup by the N Q D values it writes, the
// gradient by the N D values it reads and the V D sums it writes.  Measured: lookup
// of 100,002 ids into [25][128] fp32 173 us (7.4 TB/s written), of 16,381 tokens of
// 770 bf16 10 us; gradient over 100,002 rows and 119 ids, D = 128, 31 us a call, over
// 32,771 tokens and 50,021 x 768 67 us (floors 8 and 31).
//
// Gradient: atomics into the table would collide (a water box has two ids for
// 99 % of its rows) and sum in an order that changes from call to call.  The
// rows are put into the order of their ids by a stable radix sort of the
// (id, row) pairs, 8 bits a pass, and summed as runs of the sorted order:
//   hist_kernel      digit counts of each tile of the input
//   scatter_kernel   stable positions: every CTA sums the counts of the tiles
//                    before it (at most MAX_TILES of them) and ranks its own
//                    keys with warp matches
//   reduce_kernel    a CTA per tile of the sorted order; a row group per
//                    contiguous piece of the tile; sums of runs that end
//                    inside are written, the open ends (at most one at the
//                    head and one at the tail) are kept as partial rows.
//                    Further CTAs write zeros to the ids that do not occur
//                    (zeroing the whole table beside the sort wrote the others
//                    twice: 32,771 tokens over 50,021 x 768 73 us against 69)
//   combine_kernel   runs over several tiles: their partial rows in order
// Up to SMALL_N rows one kernel does it all: a CTA sorts the rows of its own few
// ids in shared memory.
// Every sum has a fixed order: the result repeats bit for bit.
#include <algorithm>

#include "common.cuh"
#include "embed_plan.cuh"

namespace e2f {
namespace emb {

constexpr int NT = RED_NT;

// VE consecutive elements of a row as floats (VE * sizeof(T) is 16, 4 or the
// element's size; the caller guarantees that alignment).
template <typename T, int VE> struct Vec;
template <> struct Vec<float, 4> {
  static __device__ __forceinline__ void load(const float *p, float (&v)[4]) {
    const float4 t = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Vec<float, 2> {
  static __device__ __forceinline__ void load(const float *p, float (&v)[2]) {
    v[0] = __ldg(p); v[1] = __ldg(p + 1);
  }
  static __device__ __forceinline__ void store(float *p, const float (&v)[2]) { p[0] = v[0]; p[1] = v[1]; }
};
template <> struct Vec<float, 1> {
  static __device__ __forceinline__ void load(const float *p, float (&v)[1]) { v[0] = __ldg(p); }
  static __device__ __forceinline__ void store(float *p, const float (&v)[1]) { p[0] = v[0]; }
};
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
template <> struct Vec<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p));
    v[0] = bf_lo(t.x); v[1] = bf_hi(t.x); v[2] = bf_lo(t.y); v[3] = bf_hi(t.y);
    v[4] = bf_lo(t.z); v[5] = bf_hi(t.z); v[6] = bf_lo(t.w); v[7] = bf_hi(t.w);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <> struct Vec<__nv_bfloat16, 4> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[4]) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    v[0] = bf_lo(t.x); v[1] = bf_hi(t.x); v[2] = bf_lo(t.y); v[3] = bf_hi(t.y);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
};
template <> struct Vec<__nv_bfloat16, 2> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[2]) {
    const uint32_t t = __ldg(reinterpret_cast<const uint32_t *>(p));
    v[0] = bf_lo(t); v[1] = bf_hi(t);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[2]) {
    *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v[0], v[1]);
  }
};
template <> struct Vec<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[1]) { v[0] = to_f(p[0]); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[1]) {
    p[0] = from_f<__nv_bfloat16>(v[0]);
  }
};

// VE elements of a row as loaded, and their addition to fp32 sums.
template <typename T, int VE> struct Raw {
  float v[VE];
  __device__ __forceinline__ void load(const T *p) { Vec<T, VE>::load(p, v); }
  __device__ __forceinline__ void add_to(float (&acc)[VE]) const {
#pragma unroll
    for (int k = 0; k < VE; ++k) acc[k] += v[k];
  }
};
template <> struct Raw<__nv_bfloat16, 8> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void add_to(float (&acc)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[2 * k] += bf_lo(u4w(w, k));
      acc[2 * k + 1] += bf_hi(u4w(w, k));
    }
  }
};

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
// The output is one flat run of N * VR vectors of VE elements, VR = Q D / VE;
// a CTA takes fwd_u * NT consecutive ones, so every store instruction of a
// warp is one contiguous piece.  The vector's row and place in the row advance
// by the (quotient, remainder) of NT by VR: no division per vector.
template <int VE, typename O> constexpr int fwd_u() { return VE * sizeof(O) >= 8 ? 4 : 8; }   // vectors a thread

template <typename I, typename T, typename O, int VE>
__global__ void __launch_bounds__(NT) embed_fwd_kernel(const I *__restrict__ ids, long long nvec, int VR, int DV,
                                                       const T *__restrict__ table, long long V, float scale,
                                                       O *__restrict__ out, int *err) {
  constexpr int FWD_U = fwd_u<VE, O>();
  const long long base = (long long)blockIdx.x * (FWD_U * NT);
  const long long r0 = base / VR;
  const unsigned t = (unsigned)(base - r0 * VR) + threadIdx.x;   // place counted from row r0
  long long row = r0 + t / (unsigned)VR;
  int c = (int)(t % (unsigned)VR);
  const int dq = NT / VR, dr = NT - dq * VR;
  float v[FWD_U][VE];
#pragma unroll
  for (int u = 0; u < FWD_U; ++u) {
#pragma unroll
    for (int k = 0; k < VE; ++k) v[u][k] = 0.f;
    const long long i = base + (long long)u * NT + threadIdx.x;
    if (i < nvec && c < DV) {
      const long long id = (long long)ids[row];
      if (id >= 0 && id < V) Vec<T, VE>::load(table + (size_t)id * ((size_t)DV * VE) + (size_t)c * VE, v[u]);
      else if (id != -1 && c == 0) atomicExch(err, E2F_ERR_DOMAIN);
    }
    row += dq;
    c += dr;
    if (c >= VR) { c -= VR; ++row; }
  }
#pragma unroll
  for (int u = 0; u < FWD_U; ++u) {
    const long long i = base + (long long)u * NT + threadIdx.x;
    if (i < nvec) {
      float w[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) w[k] = scale * v[u][k];
      Vec<O, VE>::store(out + (size_t)i * VE, w);
    }
  }
}

// Q = 1 and long rows: a warp per row, the id read once, eight vectors of a lane
// in flight (16,381 rows of 770 bf16: the flat kernel looks the id up for every
// vector, which costs it twice the time where a vector is two elements).
template <typename I, typename T, typename O, int VE>
__global__ void __launch_bounds__(NT) embed_row_kernel(const I *__restrict__ ids, long long N, int DV,
                                                       const T *__restrict__ table, long long V, float scale,
                                                       O *__restrict__ out, int *err) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
  if (row >= N) return;
  const long long id = (long long)ids[row];
  const bool live = id >= 0 && id < V;
  if (!live && id != -1 && lane == 0) atomicExch(err, E2F_ERR_DOMAIN);
  const T *src = table + (live ? (size_t)id * ((size_t)DV * VE) : 0);
  O *dst = out + (size_t)row * ((size_t)DV * VE);
  for (int c0 = lane; c0 < DV; c0 += 32 * U) {
    float v[U][VE];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < VE; ++k) v[u][k] = 0.f;
      if (live && c0 + 32 * u < DV) Vec<T, VE>::load(src + (size_t)(c0 + 32 * u) * VE, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 32 * u < DV) {
        float w[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) w[k] = scale * v[u][k];
        Vec<O, VE>::store(dst + (size_t)(c0 + 32 * u) * VE, w);
      }
  }
}

static bool aligned_to(const void *p, size_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }

template <typename I, typename T, typename O, int VE>
static e2f_status launch_fwd(const I *ids, int64_t N, const T *table, int64_t V, int D, float scale, int Q, O *out,
                             cudaStream_t s) {
  int *err = device_error_flag();
  if (!err) return E2F_ERR_CUDA;
  const int DV = D / VE, VR = (int)((long long)Q * DV);
  const long long nvec = (long long)N * VR;
  if (Q == 1 && DV >= 64) {
    E2F_LAUNCH((embed_row_kernel<I, T, O, VE>), (unsigned)((N + NT / 32 - 1) / (NT / 32)), NT, 0, s, ids, (long long)N, DV,
               table, (long long)V, scale, out, err);
    return E2F_OK;
  }
  constexpr int per = fwd_u<VE, O>() * NT;
  const long long grid = (nvec + per - 1) / per;
  if (grid > INT32_MAX) return E2F_ERR_UNSUPPORTED;
  E2F_LAUNCH((embed_fwd_kernel<I, T, O, VE>), (unsigned)grid, NT, 0, s, ids, nvec, VR, DV, table, (long long)V, scale,
             out, err);
  return E2F_OK;
}

// Widest vector whose loads and stores are aligned: 16 bytes of the wider type
// where they differ, else four (bf16), two or one elements.
template <typename I, typename T, typename O>
static e2f_status pick_fwd(const I *ids, int64_t N, const T *table, int64_t V, int D, float scale, int Q, O *out,
                           cudaStream_t s) {
  constexpr int W = sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4;
  if (D % W == 0 && aligned_to(table, W * sizeof(T)) && aligned_to(out, W * sizeof(O)))
    return launch_fwd<I, T, O, W>(ids, N, table, V, D, scale, Q, out, s);
  if (W == 8 && D % 4 == 0 && aligned_to(table, 4 * sizeof(T)) && aligned_to(out, 4 * sizeof(O)))
    return launch_fwd<I, T, O, 4>(ids, N, table, V, D, scale, Q, out, s);
  if (D % 2 == 0 && aligned_to(table, 2 * sizeof(T)) && aligned_to(out, 2 * sizeof(O)))
    return launch_fwd<I, T, O, 2>(ids, N, table, V, D, scale, Q, out, s);
  return launch_fwd<I, T, O, 1>(ids, N, table, V, D, scale, Q, out, s);
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, row)
// ---------------------------------------------------------------------------
constexpr int RB = 256;          // digit values of a pass

struct SortArgs {
  int N, shift, tile;            // tile: keys per CTA, a multiple of SUB
  int V;
  int tiles;
};

// Key of a row: its id, or V (behind every id) for rows that take no part.
template <typename I> __device__ __forceinline__ uint32_t key_of(const I *ids, int n, int V) {
  const long long id = (long long)ids[n];
  return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
}

// FIRST: the keys are read from the ids, the rows are 0, 1, 2, ...
template <typename I, bool FIRST>
__global__ void __launch_bounds__(NT) hist_kernel(SortArgs a, const I *__restrict__ ids,
                                                  const uint32_t *__restrict__ keys, int *__restrict__ hist, int *err) {
  __shared__ int h[RB];
  after_previous();
  h[threadIdx.x] = 0;
  __syncthreads();
  const long long lo = (long long)blockIdx.x * a.tile;
  const long long hi = lo + a.tile < a.N ? lo + a.tile : a.N;
  for (long long i = lo + threadIdx.x; i < hi; i += NT) {
    uint32_t k;
    if (FIRST) {
      k = key_of(ids, (int)i, a.V);
      if (k == (uint32_t)a.V && (long long)ids[i] != -1) atomicExch(err, E2F_ERR_DOMAIN);
    } else {
      k = keys[i];
    }
    atomicAdd(&h[(k >> a.shift) & (RB - 1)], 1);
  }
  __syncthreads();
  hist[blockIdx.x * RB + threadIdx.x] = h[threadIdx.x];
}

template <typename I, bool FIRST>
__global__ void __launch_bounds__(NT) scatter_kernel(SortArgs a, const I *__restrict__ ids,
                                                     const uint32_t *__restrict__ keys, const int *__restrict__ rows,
                                                     const int *__restrict__ hist, uint32_t *__restrict__ keys_out,
                                                     int *__restrict__ rows_out) {
  constexpr int NW = NT / 32, PER = SUB / NT;
  __shared__ int cnt[NW][RB];   // keys of the digit in the warps before, then the warp's running position
  __shared__ int scan[RB];
  __shared__ int base[RB];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  after_previous();
  // base[d]: keys of smaller digits anywhere, and of digit d in earlier tiles
  {
    int before = 0, total = 0;
#pragma unroll 8
    for (int b = 0; b < a.tiles; ++b) {
      const int c = hist[b * RB + t];
      if (b < (int)blockIdx.x) before += c;
      total += c;
    }
    scan[t] = total;
    __syncthreads();
    for (int o = 1; o < RB; o <<= 1) {
      const int v = t >= o ? scan[t - o] : 0;
      __syncthreads();
      scan[t] += v;
      __syncthreads();
    }
    base[t] = scan[t] - total + before;
  }
  const long long lo = (long long)blockIdx.x * a.tile;
  const long long hi = lo + a.tile < a.N ? lo + a.tile : a.N;
  for (long long s0 = lo; s0 < hi; s0 += SUB) {
#pragma unroll
    for (int w = 0; w < NW; ++w) cnt[w][t] = 0;
    __syncthreads();
    // warp w ranks the keys [s0 + w * SUB / NW, + SUB / NW), 32 at a time
    uint32_t k[PER];
    int rank[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const long long i = s0 + warp * (SUB / NW) + j * 32 + lane;
      const bool live = i < hi;
      k[j] = 0;
      if (live) k[j] = FIRST ? key_of(ids, (int)i, a.V) : keys[i];
      const uint32_t d = live ? (k[j] >> a.shift) & (RB - 1) : (uint32_t)RB;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      int before = 0;
      if (live) before = cnt[warp][d];
      __syncwarp();
      rank[j] = before + __popc(same & ((1u << lane) - 1u));
      if (live && (same >> lane) == 1u) cnt[warp][d] = before + __popc(same);   // the last lane of the digit
      __syncwarp();
    }
    __syncthreads();
    {
      int run = base[t];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int c = cnt[w][t];
        cnt[w][t] = run;
        run += c;
      }
      base[t] = run;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const long long i = s0 + warp * (SUB / NW) + j * 32 + lane;
      if (i < hi) {
        const int p = cnt[warp][(k[j] >> a.shift) & (RB - 1)] + rank[j];
        keys_out[p] = k[j];
        rows_out[p] = FIRST ? (int)i : rows[i];
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// sums over runs of equal keys
// ---------------------------------------------------------------------------
// CL lanes over the columns of a block of CL * VE, RG = NT / CL row groups; a
// tile is R consecutive places of the sorted order, a group has R / RG of them.
struct RedArgs {
  int N, V, D, CL, R;
  long long ld;           // elements between rows of grad_out
  float scale;
  int accumulate;
  bool gvec;              // rows of grad start on 16-byte boundaries
  const uint32_t *keys;   // sorted
  const int *rows;
  float *grad;            // [V][D]
  float *head, *tail;     // [tiles][D] partial rows of runs that cross the tile's start / end
  int tiles;
};

// VE floats to p: 16 bytes at a time where the row starts on such a boundary.
template <int VE> __device__ __forceinline__ void put_row(float *p, const float (&v)[VE], bool vec) {
  if (VE >= 4 && vec) {
#pragma unroll
    for (int k = 0; k < VE / 4; ++k)
      reinterpret_cast<float4 *>(p)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < VE; ++k) p[k] = v[k];
  }
}
// The sum of an id's rows (columns col .. col + VE, all inside: VE divides D).
template <int VE> __device__ __forceinline__ void write_sum(const RedArgs &a, uint32_t key, int col, const float (&acc)[VE]) {
  float *p = a.grad + (size_t)key * a.D + col;
  float v[VE];
#pragma unroll
  for (int k = 0; k < VE; ++k) v[k] = a.accumulate ? p[k] + a.scale * acc[k] : a.scale * acc[k];
  put_row<VE>(p, v, a.gvec);
}

// First place of the sorted keys with a key >= v, by a whole warp: 32 probes a step.
__device__ __forceinline__ int lower_bound_warp(const uint32_t *keys, int n, uint32_t v, int lane) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = probe_step(lo, hi), p = probe_at(lo, step, lane);
    const uint32_t ge = __ballot_sync(0xffffffffu, p >= hi || keys[p] >= v);
    narrow(lo, hi, step, ge ? __ffs(ge) - 1 : 32);
  }
  return lo;
}

// Zeros to those of the ids v0 .. v0 + ZROWS that do not occur.
__device__ __forceinline__ void zero_absent(const RedArgs &a, long long v0, int *sm) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int nv = (int)min((long long)ZROWS, a.V - v0);
  if (warp < 2) {
    const int p = lower_bound_warp(a.keys, a.N, (uint32_t)(v0 + (warp ? nv : 0)), lane);
    if (lane == 0) sm[ZROWS + warp] = p;
  }
  __syncthreads();
  if (t < nv) {   // among the keys of these ids
    const uint32_t v = (uint32_t)(v0 + t);
    int lo = sm[ZROWS], hi = sm[ZROWS + 1];
    const int end = hi;
    while (lo < hi) {
      const int mid = lo + ((hi - lo) >> 1);
      if (a.keys[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    sm[t] = lo == end || a.keys[lo] != v;
  }
  __syncthreads();
  for (int r = warp; r < nv; r += NT / 32) {
    if (!sm[r]) continue;
    float *p = a.grad + (size_t)(v0 + r) * a.D;
    if (a.gvec) {
      for (int c = lane; c < a.D / 4; c += 32) reinterpret_cast<float4 *>(p)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int c = lane; c < a.D; c += 32) p[c] = 0.f;
    }
  }
}

template <typename T, int VE>
__global__ void __launch_bounds__(NT, RED_CTAS) reduce_kernel(RedArgs a, const T *__restrict__ g) {
  extern __shared__ int sm[];
  const int t = threadIdx.x;
  after_previous();
  if ((int)blockIdx.x >= a.tiles) {
    if (blockIdx.y == 0) zero_absent(a, (long long)((int)blockIdx.x - a.tiles) * ZROWS, sm);
    return;
  }
  const int CL = a.CL, RG = NT / CL, R = a.R, G = R / RG;
  uint32_t *skey = reinterpret_cast<uint32_t *>(sm);      // [R + 2]: key before, the tile's, key behind
  int *srow = sm + R + 2;                                 // [R]
  float *shead = reinterpret_cast<float *>(sm + 2 * R + 2);   // [RG][CL * VE]
  float *stail = shead + NT * VE;
  int *sflag = sm + 2 * R + 2 + 2 * NT * VE;              // [RG]
  uint32_t *sends = reinterpret_cast<uint32_t *>(sflag + RG);   // [R / 32 + 1]: bit i: a run ends at place i
  const int p0 = blockIdx.x * R;
  const int np = a.N - p0 < R ? a.N - p0 : R;
  const uint32_t NOKEY = 0xffffffffu;                     // no id: V < 2^31
  int valid = 0;
  for (int i = t; i < np + 2; i += NT) {
    const long long p = (long long)p0 + i - 1;
    const uint32_t k = p >= 0 && p < a.N ? a.keys[p] : NOKEY;
    skey[i] = k;
    valid += i >= 1 && i <= np && k < (uint32_t)a.V;
  }
  for (int i = t; i < np; i += NT) srow[i] = a.rows[p0 + i];
  // rows that take no part are sorted behind the others
  __shared__ int nvalid;
  if (t == 0) nvalid = 0;
  __syncthreads();
  valid = warp_sum_i(valid);
  if ((t & 31) == 0 && valid) atomicAdd(&nvalid, valid);
  const uint32_t *key = skey + 1;
  for (int i0 = t & ~31; i0 < R + 32; i0 += NT) {
    const int i = i0 + (t & 31);
    const uint32_t e = __ballot_sync(0xffffffffu, i >= np || key[i] != key[i + 1]);
    if ((t & 31) == 0) sends[i0 >> 5] = e;
  }
  __syncthreads();
  const int n = nvalid;
  const int cl = t % CL, rg = t / CL;
  const int col = (blockIdx.y * CL + cl) * VE;
  const bool in = col < a.D;
  // group pass: places [i0, i1), U rows being added while the next U are on their way
  {
    const int i0 = rg * G < n ? rg * G : n, i1 = i0 + G < n ? i0 + G : n;
    const uint32_t ends = __funnelshift_r(sends[i0 >> 5], sends[(i0 >> 5) + 1], i0 & 31);
    float acc[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) acc[k] = 0.f;
    bool fresh = i0 < i1 && key[i0] != key[i0 - 1];   // the open run started inside this group
    int flag = 0;          // 1: head partial, 2: it runs through the group, 4: tail partial
    constexpr int U = VE >= 4 ? 4 : 8;
    const T *gc = g + (in ? col : 0);
    Raw<T, VE> cur[U], nxt[U];
    auto fetch = [&](Raw<T, VE> (&r)[U], int i) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < i1) r[u].load(gc + (size_t)srow[i + u] * a.ld);
    };
    fetch(cur, i0);
    for (int i = i0; i < i1; i += U) {
      fetch(nxt, i + U);
      const uint32_t eb = ends >> (i - i0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u < i1) {
          cur[u].add_to(acc);
          if (eb >> u & 1) {   // the run ends here
            if (fresh) {
              if (in) write_sum<VE>(a, key[i + u], col, acc);
            } else {
              flag |= 1;
#pragma unroll
              for (int k = 0; k < VE; ++k) shead[(rg * CL + cl) * VE + k] = acc[k];
            }
            fresh = true;
#pragma unroll
            for (int k = 0; k < VE; ++k) acc[k] = 0.f;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }
    if (i0 < i1 && !(ends >> (i1 - 1 - i0) & 1)) {   // open at the group's end
      float *dst = fresh ? stail : shead;
      flag |= fresh ? 4 : 3;
#pragma unroll
      for (int k = 0; k < VE; ++k) dst[(rg * CL + cl) * VE + k] = acc[k];
    }
    if (cl == 0) sflag[rg] = flag;
  }
  __syncthreads();
  // join the groups in order
  if (rg == 0 && in) {
    float acc[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) acc[k] = 0.f;
    bool fresh = false, open = false;
    for (int q = 0; q < RG && q * G < n; ++q) {
      const int f = sflag[q];
      const int i1 = (q + 1) * G < n ? (q + 1) * G : n;
      if (f & 1) {
        const float *h = shead + (q * CL + cl) * VE;
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] += h[k];
        open = true;
        if (!(f & 2)) {   // ends in this group
          const uint32_t kk = key[q * G];
          if (!fresh) put_row<VE>(a.head + (size_t)blockIdx.x * a.D + col, acc, true);
          else write_sum<VE>(a, kk, col, acc);
          open = false;
        }
      }
      if (f & 4) {
        const float *h = stail + (q * CL + cl) * VE;
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] = h[k];
        open = fresh = true;
      }
      if (i1 == n && open) {   // runs on into the next tile
        put_row<VE>((fresh ? a.tail : a.head) + (size_t)blockIdx.x * a.D + col, acc, true);
      }
    }
  }
}

// Runs over several tiles.  A warp looks at one tile: where a run starts inside
// the tile and goes on behind it, it adds the tail row and the head rows of the
// tiles up to the one where the run ends.  Runs over more than 32 tiles are left
// to the whole CTA, JG head rows side by side.
constexpr int JG = 32;
__global__ void __launch_bounds__(32 * JG) combine_kernel(RedArgs a) {
  __shared__ float part[JG][32];
  __shared__ int todo[JG];
  __shared__ int last;
  const int t = threadIdx.x, lane = t & 31, jg = t >> 5;
  after_previous();
  {
    const int b = blockIdx.x * JG + jg;
    bool act = false;
    uint32_t kk = 0;
    if (b < a.tiles - 1) {
      const long long pe = ((long long)b + 1) * a.R, p0 = pe - a.R;   // the tile is [p0, pe)
      kk = a.keys[pe - 1];
      const uint32_t behind = a.keys[pe], before = p0 > 0 ? a.keys[p0 - 1] : 0xffffffffu;
      act = behind == kk && before != kk && kk < (uint32_t)a.V;
    }
    bool lng = false;
    if (act) {   // uniform in the warp
      const int q = b + 1 + lane;
      // the first tile behind that does not end with the id, and whether it starts with it
      const bool ends = q >= a.tiles - 1 || a.keys[((long long)q + 1) * a.R - 1] != kk;
      const bool starts = q < a.tiles && a.keys[(long long)q * a.R] == kk;
      const uint32_t e = __ballot_sync(0xffffffffu, ends), f = __ballot_sync(0xffffffffu, starts);
      lng = e == 0;
      if (!lng) {
        const int i = __ffs(e) - 1, n = (f >> i & 1) ? i + 1 : i;   // head rows
        for (int col = blockIdx.y * 32 + lane; col < a.D; col += gridDim.y * 32) {
          float s[1] = {a.tail[(size_t)b * a.D + col]};
#pragma unroll 4
          for (int k = 1; k <= n; ++k) s[0] += a.head[(size_t)(b + k) * a.D + col];
          write_sum<1>(a, kk, col, s);
        }
      }
    }
    if (lane == 0) todo[jg] = lng;
  }
  __syncthreads();
  for (int j = 0; j < JG; ++j) {
    if (!todo[j]) continue;
    const int b = blockIdx.x * JG + j;
    const uint32_t kk = a.keys[((long long)b + 1) * a.R - 1];
    for (int q0 = b + 1;; q0 += 32 * JG) {
      const int q = q0 + t;
      const bool ends = q >= a.tiles - 1 || a.keys[((long long)q + 1) * a.R - 1] != kk;
      if (t == 0) last = INT32_MAX;
      __syncthreads();
      if (ends) atomicMin(&last, q);
      __syncthreads();
      if (last != INT32_MAX) break;
    }
    int tl = last;
    if (a.keys[(long long)tl * a.R] != kk) --tl;   // it may not even start with the id
    for (int c0 = blockIdx.y * 32; c0 < a.D; c0 += gridDim.y * 32) {
      const int col = c0 + lane;
      float s = 0.f;
      if (col < a.D) {
        if (jg == 0) s = a.tail[(size_t)b * a.D + col];
#pragma unroll 16
        for (int q = b + 1 + jg; q <= tl; q += JG) s += a.head[(size_t)q * a.D + col];
      }
      part[jg][lane] = s;
      __syncthreads();
      if (jg == 0 && col < a.D) {
        float one[1] = {part[0][lane]};
#pragma unroll
        for (int i = 1; i < JG; ++i) one[0] += part[i][lane];
        write_sum<1>(a, kk, col, one);
      }
      __syncthreads();
    }
  }
}

template <typename T, int VE>
static e2f_status launch_reduce(RedArgs a, int zero, const T *g, cudaStream_t s) {
  const int dv = (a.D + VE - 1) / VE;
  const int RG = NT / a.CL;
  const size_t smem = sizeof(int) * (size_t)(2 * a.R + 2 + 2 * NT * VE + RG + a.R / 32 + 2);
  dim3 grid((unsigned)a.tiles + (unsigned)zero, (unsigned)((dv + a.CL - 1) / a.CL));
  E2F_LAUNCH_AFTER((reduce_kernel<T, VE>), grid, NT, smem, s, a, g);
  if (a.tiles > 1) {
    dim3 cg((unsigned)((a.tiles - 1 + JG - 1) / JG), (unsigned)std::min(64, (a.D + 31) / 32));
    E2F_LAUNCH_AFTER(combine_kernel, cg, 32 * JG, 0, s, a);
  }
  return E2F_OK;
}

// ---------------------------------------------------------------------------
// Few rows: one kernel.  A CTA has the ids [v0, v0 + W) and a block of columns:
// it ranks the rows of its ids as a radix pass does (digit: id - v0), keeps them
// sorted in shared memory and sums each id's rows, a warp to a short list, the
// whole CTA to a long one.  No scratch, one launch: latency is what it costs.
// ---------------------------------------------------------------------------
constexpr int SMALL_N = 1024, SMALL_W = 256, LONG_LIST = 64;

template <typename I, typename T, int VE>
__global__ void __launch_bounds__(NT) small_kernel(RedArgs a, int W, const I *__restrict__ ids, const T *__restrict__ g,
                                                   int *err) {
  constexpr int NW = NT / 32;
  __shared__ int cnt[NW][SMALL_W];
  __shared__ int start[SMALL_W + 1];
  __shared__ int srow[SMALL_N];
  __shared__ float part[NW][32 * VE];
  __shared__ int longs[SMALL_N / LONG_LIST], nlong;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int v0 = blockIdx.x * W, nw = min(W, a.V - v0);
  for (int i = t; i < NW * SMALL_W; i += NT) cnt[0][i] = 0;
  __syncthreads();
  // warp w ranks the rows [w per, (w + 1) per)
  constexpr int PER = SMALL_N / NT;
  const int per = (a.N + NW * 32 - 1) / (NW * 32) * 32;
  int key[PER], rank[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = warp * per + j * 32 + lane;
    key[j] = -1;
    if (j * 32 < per && i < a.N) {
      const long long id = (long long)ids[i];
      if (id >= v0 && id < v0 + nw) key[j] = (int)(id - v0);
      else if ((id < -1 || id >= a.V) && blockIdx.x == 0 && blockIdx.y == 0) atomicExch(err, E2F_ERR_DOMAIN);
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    rank[j] = 0;
    if (j * 32 >= per || !__any_sync(0xffffffffu, key[j] >= 0)) continue;
    const uint32_t same = __match_any_sync(0xffffffffu, key[j]);
    int before = 0;
    if (key[j] >= 0) before = cnt[warp][key[j]];
    __syncwarp();
    rank[j] = before + __popc(same & ((1u << lane) - 1u));
    if (key[j] >= 0 && (same >> lane) == 1u) cnt[warp][key[j]] = before + __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // start[d]: rows of smaller ids; cnt[w][d]: first place of warp w's rows of id d
  {
    int total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) total += cnt[w][t];
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    __shared__ int wsum[NW];
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int off = 0;
    for (int w = 0; w < warp; ++w) off += wsum[w];
    int run = off + incl - total;
    start[t] = run;
    if (t == SMALL_W - 1) start[SMALL_W] = run + total;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c = cnt[w][t];
      cnt[w][t] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (key[j] >= 0) srow[cnt[warp][key[j]] + rank[j]] = warp * per + j * 32 + lane;
  __syncthreads();
  // CL lanes over the columns, S = 32 / CL rows side by side
  const int CL = a.CL, S = 32 / CL, cl = lane % CL, sub = lane / CL;
  const int col = (blockIdx.y * CL + cl) * VE;
  const bool in = col < a.D;
  auto warp_rows = [&](int i0, int i1, float (&acc)[VE]) {
#pragma unroll
    for (int k = 0; k < VE; ++k) acc[k] = 0.f;
    constexpr int U = VE == 8 ? 4 : 8;
    for (int i = i0 + sub; i < i1; i += U * S) {
      float v[U][VE];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < VE; ++k) v[u][k] = 0.f;
        if (i + u * S < i1 && in) Vec<T, VE>::load(g + (size_t)srow[i + u * S] * a.ld + col, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] += v[u][k];
    }
    for (int o = CL; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < VE; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
  };
  // short lists, and zeros for the ids that do not occur
  const int c0 = blockIdx.y * CL * VE, cw = min(CL * VE, a.D - c0);
  if (t == 0) nlong = 0;
  __syncthreads();
  float acc[VE];
  for (int d = warp; d < nw; d += NW) {
    const int i0 = start[d], n = start[d + 1] - i0;
    if (n == 0) {
      if (a.accumulate) continue;
      float *p = a.grad + (size_t)(v0 + d) * a.D + c0;
      if (VE >= 4 && a.gvec)
        for (int c = lane; c < cw / 4; c += 32) reinterpret_cast<float4 *>(p)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      else
        for (int c = lane; c < cw; c += 32) p[c] = 0.f;
    } else if (n <= LONG_LIST) {
      warp_rows(i0, i0 + n, acc);
      if (sub == 0 && in) write_sum<VE>(a, (uint32_t)(v0 + d), col, acc);
    } else if (lane == 0) {
      longs[atomicAdd(&nlong, 1)] = d;
    }
  }
  __syncthreads();
  for (int l = 0; l < nlong; ++l) {   // (any order: each id's sum stands alone)
    const int d = longs[l], n = start[d + 1] - start[d];
    const int piece = (n + NW - 1) / NW, i0 = start[d] + min(n, warp * piece), i1 = start[d] + min(n, (warp + 1) * piece);
    warp_rows(i0, i1, acc);
    __syncthreads();
    if (sub == 0)
#pragma unroll
      for (int k = 0; k < VE; ++k) part[warp][cl * VE + k] = acc[k];
    __syncthreads();
    if (warp == 0 && sub == 0 && in) {
#pragma unroll
      for (int w = 1; w < NW; ++w)
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] += part[w][cl * VE + k];
      write_sum<VE>(a, (uint32_t)(v0 + d), col, acc);
    }
  }
}

template <typename I, typename T, int VE>
static e2f_status launch_small(RedArgs a, const I *ids, const T *g, int *err, cudaStream_t s) {
  const int dv = (a.D + VE - 1) / VE;
  // Enough CTAs for the device: ids first, then blocks of eight vectors of
  // columns instead of 32 where there are few ids.
  const int W = std::min(SMALL_W, std::max(1, (a.V + 591) / 592));
  const int ctas = (a.V + W - 1) / W;
  const int widest = ctas * ((dv + 31) / 32) < 296 ? 8 : 32;
  a.CL = 1;
  while (a.CL < widest && a.CL < dv) a.CL <<= 1;
  dim3 grid((unsigned)ctas, (unsigned)((dv + a.CL - 1) / a.CL));
  E2F_LAUNCH((small_kernel<I, T, VE>), grid, NT, 0, s, a, W, ids, g, err);
  return E2F_OK;
}

template <typename I, typename T>
static e2f_status backward(const I *ids, int64_t N64, const T *g, int64_t V, int D, float scale, int Q, float *grad,
                           int accumulate, cudaStream_t s) {
  const int N = (int)N64;
  if (N == 0) {
    if (!accumulate) E2F_CUDA_TRY(cudaMemsetAsync(grad, 0, sizeof(float) * (size_t)V * D, s));
    return E2F_OK;
  }
  int *err = device_error_flag();
  if (!err) return E2F_ERR_CUDA;
  const long long ld = (long long)Q * D;
  constexpr int W = 16 / (int)sizeof(T);
  const int VE = D % W == 0 && aligned_to(g, 16) ? W : (D % 2 == 0 && aligned_to(g, 2 * sizeof(T)) ? 2 : 1);
  RedArgs a{};
  a.N = N; a.V = (int)V; a.D = D; a.ld = ld; a.scale = scale; a.accumulate = accumulate; a.grad = grad;
  a.gvec = D % 4 == 0 && aligned_to(grad, 16);
  if (N <= SMALL_N) {
    if (VE == W) return launch_small<I, T, W>(a, ids, g, err, s);
    if (VE == 2) return launch_small<I, T, 2>(a, ids, g, err, s);
    return launch_small<I, T, 1>(a, ids, g, err, s);
  }
  const RunPlan rp = run_plan(N, V, (D + VE - 1) / VE);
  a.CL = rp.CL;
  a.R = rp.R;
  a.tiles = rp.tiles;
  const int zero = accumulate ? 0 : rp.zero;
  const SortPlan sp = sort_plan(N, V);
  SortArgs sa{};
  sa.N = N; sa.V = (int)V; sa.tile = sp.tile; sa.tiles = sp.tiles;
  const int st = sp.tiles, passes = sp.passes;
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  const size_t kb = up(sizeof(int) * (size_t)N), pb = up(sizeof(float) * (size_t)a.tiles * D);
  Scratch ws;
  E2F_CUDA_TRY(ws.alloc(4 * kb + up(sizeof(int) * (size_t)st * RB) + 2 * pb, s));
  char *w = ws.as<char>();
  uint32_t *k0 = reinterpret_cast<uint32_t *>(w), *k1 = reinterpret_cast<uint32_t *>(w + kb);
  int *q0 = reinterpret_cast<int *>(w + 2 * kb), *q1 = reinterpret_cast<int *>(w + 3 * kb);
  a.head = reinterpret_cast<float *>(w + 4 * kb);
  a.tail = reinterpret_cast<float *>(w + 4 * kb + pb);
  int *hist = reinterpret_cast<int *>(w + 4 * kb + 2 * pb);
  E2F_LAUNCH((hist_kernel<I, true>), st, NT, 0, s, sa, ids, nullptr, hist, err);
  E2F_LAUNCH_AFTER((scatter_kernel<I, true>), st, NT, 0, s, sa, ids, nullptr, nullptr, hist, k0, q0);
  for (int pass = 1; pass < passes; ++pass) {
    sa.shift = 8 * pass;
    E2F_LAUNCH_AFTER((hist_kernel<I, false>), st, NT, 0, s, sa, nullptr, k0, hist, err);
    E2F_LAUNCH_AFTER((scatter_kernel<I, false>), st, NT, 0, s, sa, nullptr, k0, q0, hist, k1, q1);
    std::swap(k0, k1);
    std::swap(q0, q1);
  }
  a.keys = k0;
  a.rows = q0;
  if (VE == W) return launch_reduce<T, W>(a, zero, g, s);
  if (VE == 2) return launch_reduce<T, 2>(a, zero, g, s);
  return launch_reduce<T, 1>(a, zero, g, s);
}

template <typename I>
static e2f_status forward_i(const I *ids, int64_t N, const void *table, int dtype, int64_t V, int D, float scale, int Q,
                            void *out, int out_dtype, cudaStream_t s) {
  if (dtype == E2F_F32) {
    const float *t = static_cast<const float *>(table);
    return out_dtype == E2F_F32 ? pick_fwd<I, float, float>(ids, N, t, V, D, scale, Q, static_cast<float *>(out), s)
                                : pick_fwd<I, float, __nv_bfloat16>(ids, N, t, V, D, scale, Q,
                                                                    static_cast<__nv_bfloat16 *>(out), s);
  }
  const __nv_bfloat16 *t = static_cast<const __nv_bfloat16 *>(table);
  return out_dtype == E2F_F32
             ? pick_fwd<I, __nv_bfloat16, float>(ids, N, t, V, D, scale, Q, static_cast<float *>(out), s)
             : pick_fwd<I, __nv_bfloat16, __nv_bfloat16>(ids, N, t, V, D, scale, Q, static_cast<__nv_bfloat16 *>(out), s);
}

template <typename I>
static e2f_status backward_i(const I *ids, int64_t N, const void *g, int dtype, int64_t V, int D, float scale, int Q,
                             float *grad, int accumulate, cudaStream_t s) {
  if (dtype == E2F_F32) return backward<I, float>(ids, N, static_cast<const float *>(g), V, D, scale, Q, grad, accumulate, s);
  return backward<I, __nv_bfloat16>(ids, N, static_cast<const __nv_bfloat16 *>(g), V, D, scale, Q, grad, accumulate, s);
}

}  // namespace emb

e2f_status embed_forward_impl(const void *ids, int id_type, int64_t N, const void *table, int dtype, int64_t V, int D,
                              float scale, int Q, void *out, int out_dtype, cudaStream_t s) {
  if (id_type == E2F_I32)
    return emb::forward_i(static_cast<const int32_t *>(ids), N, table, dtype, V, D, scale, Q, out, out_dtype, s);
  return emb::forward_i(static_cast<const int64_t *>(ids), N, table, dtype, V, D, scale, Q, out, out_dtype, s);
}

e2f_status embed_backward_impl(const void *ids, int id_type, int64_t N, const void *grad_out, int dtype, int64_t V, int D,
                               float scale, int Q, float *grad_table, int accumulate, cudaStream_t s) {
  if (id_type == E2F_I32)
    return emb::backward_i(static_cast<const int32_t *>(ids), N, grad_out, dtype, V, D, scale, Q, grad_table, accumulate, s);
  return emb::backward_i(static_cast<const int64_t *>(ids), N, grad_out, dtype, V, D, scale, Q, grad_table, accumulate, s);
}

}  // namespace e2f
