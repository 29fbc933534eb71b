// Scaled embedding lookup (ids -> the l = 0 rows of node features) and its
// gradient by sorted ids.
//
//   out[n][0][:] = scale * table[id_n],  out[n][q > 0][:] = 0
//   grad_table[v][:] = scale * sum over {n : id_n = v} of grad_out[n][0][:]
//
// Both are bound by HBM: the lookup by the N Q D values it writes, the
// gradient by the N D values it reads and the V D sums it writes.
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
//                    Further CTAs write zeros to the ids that do not occur.
//   combine_kernel   runs over several tiles: their partial rows in order
// Every sum has a fixed order: the result repeats bit for bit.
#include <algorithm>

#include "common.cuh"

namespace e2f {
namespace emb {

constexpr int NT = 256;

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

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
// The output is one flat run of N * VR vectors of VE elements, VR = Q D / VE;
// a CTA takes FWD_U * NT consecutive ones, so every store instruction of a
// warp is one contiguous piece.  The vector's row and place in the row advance
// by the (quotient, remainder) of NT by VR: no division per vector.
constexpr int FWD_U = 4;

template <typename I, typename T, typename O, int VE>
__global__ void __launch_bounds__(NT) embed_fwd_kernel(const I *__restrict__ ids, long long nvec, int VR, int DV,
                                                       const T *__restrict__ table, long long V, float scale,
                                                       O *__restrict__ out, int *err) {
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

static bool aligned_to(const void *p, size_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }

template <typename I, typename T, typename O, int VE>
static e2f_status launch_fwd(const I *ids, int64_t N, const T *table, int64_t V, int D, float scale, int Q, O *out,
                             cudaStream_t s) {
  int *err = device_error_flag();
  if (!err) return E2F_ERR_CUDA;
  const int DV = D / VE, VR = (int)((long long)Q * DV);
  const long long nvec = (long long)N * VR;
  const long long grid = (nvec + FWD_U * NT - 1) / (FWD_U * NT);
  if (grid > INT32_MAX) return E2F_ERR_UNSUPPORTED;
  E2F_LAUNCH((embed_fwd_kernel<I, T, O, VE>), (unsigned)grid, NT, 0, s, ids, nvec, VR, DV, table, (long long)V, scale,
             out, err);
  return E2F_OK;
}

// Widest vector whose loads and stores are aligned: 16 bytes of the narrower
// type, else two or one elements.
template <typename I, typename T, typename O>
static e2f_status pick_fwd(const I *ids, int64_t N, const T *table, int64_t V, int D, float scale, int Q, O *out,
                           cudaStream_t s) {
  constexpr int W = sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4;
  if (D % W == 0 && aligned_to(table, W * sizeof(T)) && aligned_to(out, W * sizeof(O)))
    return launch_fwd<I, T, O, W>(ids, N, table, V, D, scale, Q, out, s);
  if (D % 2 == 0 && aligned_to(table, 2 * sizeof(T)) && aligned_to(out, 2 * sizeof(O)))
    return launch_fwd<I, T, O, 2>(ids, N, table, V, D, scale, Q, out, s);
  return launch_fwd<I, T, O, 1>(ids, N, table, V, D, scale, Q, out, s);
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, row)
// ---------------------------------------------------------------------------
constexpr int RB = 256;          // digit values of a pass
constexpr int SUB = 2048;        // keys a CTA ranks at a time: 8 warps x 256
constexpr int MAX_TILES = 128;   // CTAs of a pass; longer inputs give each more keys

struct SortArgs {
  int N, shift, tile;            // tile: keys per CTA, a multiple of SUB
  int V;
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
  // base[d]: keys of smaller digits anywhere, and of digit d in earlier tiles
  {
    int before = 0, total = 0;
    for (int b = 0; b < (int)gridDim.x; ++b) {
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
  const uint32_t *keys;   // sorted
  const int *rows;
  float *grad;            // [V][D]
  float *head, *tail;     // [tiles][D] partial rows of runs that cross the tile's start / end
  int tiles;
};

template <int VE> __device__ __forceinline__ void write_sum(const RedArgs &a, uint32_t key, int col, const float (&acc)[VE]) {
  float *p = a.grad + (size_t)key * a.D + col;
#pragma unroll
  for (int k = 0; k < VE; ++k)
    if (col + k < a.D) p[k] = a.accumulate ? p[k] + a.scale * acc[k] : a.scale * acc[k];
}

constexpr int ZROWS = 32;   // ids a zero-writing CTA looks after

template <typename T, int VE>
__global__ void __launch_bounds__(NT) reduce_kernel(RedArgs a, const T *__restrict__ g) {
  extern __shared__ int sm[];
  const int t = threadIdx.x;
  if ((int)blockIdx.x >= a.tiles) {
    // ids v0 .. v0 + ZROWS that do not occur: zeros (first column block only
    // launches these CTAs with blockIdx.y == 0 doing the whole row)
    if (blockIdx.y != 0) return;
    const long long v0 = (long long)((int)blockIdx.x - a.tiles) * ZROWS;
    if (t < ZROWS) {
      int absent = 0;
      if (v0 + t < a.V) {
        const uint32_t v = (uint32_t)(v0 + t);
        int lo = 0, hi = a.N;   // first place with key >= v
        while (lo < hi) {
          const int mid = lo + ((hi - lo) >> 1);
          if (a.keys[mid] < v) lo = mid + 1;
          else hi = mid;
        }
        absent = lo == a.N || a.keys[lo] != v;
      }
      sm[t] = absent;
    }
    __syncthreads();
    for (int r = 0; r < ZROWS; ++r)
      if (sm[r]) {
        float *p = a.grad + (size_t)(v0 + r) * a.D;
        if ((a.D & 3) == 0 && (reinterpret_cast<uintptr_t>(a.grad) & 15) == 0) {
          for (int c = t; c < a.D / 4; c += NT) reinterpret_cast<float4 *>(p)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
          for (int c = t; c < a.D; c += NT) p[c] = 0.f;
        }
      }
    return;
  }
  const int CL = a.CL, RG = NT / CL, R = a.R, G = R / RG;
  uint32_t *skey = reinterpret_cast<uint32_t *>(sm);      // [R + 2]: key before, the tile's, key behind
  int *srow = sm + R + 2;                                 // [R]
  float *shead = reinterpret_cast<float *>(sm + 2 * R + 2);   // [RG][CL * VE]
  float *stail = shead + NT * VE;
  int *sflag = sm + 2 * R + 2 + 2 * NT * VE;              // [RG]
  const int p0 = blockIdx.x * R;
  const int n = a.N - p0 < R ? a.N - p0 : R;
  const uint32_t NOKEY = 0xffffffffu;                     // no id: V < 2^31
  for (int i = t; i < n + 2; i += NT) {
    const long long p = (long long)p0 + i - 1;
    skey[i] = p >= 0 && p < a.N ? a.keys[p] : NOKEY;
  }
  for (int i = t; i < n; i += NT) srow[i] = a.rows[p0 + i];
  __syncthreads();
  const int cl = t % CL, rg = t / CL;
  const int col = (blockIdx.y * CL + cl) * VE;
  const bool in = col < a.D;
  const uint32_t *key = skey + 1;
  // group pass: places [i0, i1)
  {
    const int i0 = rg * G < n ? rg * G : n, i1 = i0 + G < n ? i0 + G : n;
    float acc[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) acc[k] = 0.f;
    bool fresh = false;    // the open run started inside this group
    int flag = 0;          // 1: head partial, 2: it runs through the group, 4: tail partial
    if (i0 < i1) fresh = key[i0] != key[i0 - 1];
    constexpr int U = 8;
    for (int i = i0; i < i1; i += U) {
      float v[U][VE];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < VE; ++k) v[u][k] = 0.f;
        if (i + u < i1 && in && key[i + u] < (uint32_t)a.V)
          Vec<T, VE>::load(g + (size_t)srow[i + u] * a.ld + col, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u >= i1) break;
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] += v[u][k];
        const uint32_t kk = key[i + u];
        if (kk != key[i + u + 1]) {   // the run ends here
          if (fresh) {
            if (in && kk < (uint32_t)a.V) write_sum<VE>(a, kk, col, acc);
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
    if (i0 < i1 && key[i1 - 1] == key[i1]) {   // open at the group's end
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
          if (!fresh) {
#pragma unroll
            for (int k = 0; k < VE; ++k)
              if (col + k < a.D) a.head[(size_t)blockIdx.x * a.D + col + k] = acc[k];
          } else if (kk < (uint32_t)a.V) {
            write_sum<VE>(a, kk, col, acc);
          }
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
        float *dst = fresh ? a.tail : a.head;
#pragma unroll
        for (int k = 0; k < VE; ++k)
          if (col + k < a.D) dst[(size_t)blockIdx.x * a.D + col + k] = acc[k];
      }
    }
  }
}

// Runs over several tiles.  CTA (tile, column block) acts where a run starts
// inside the tile and goes on behind it: its tail row, then the head rows of
// the tiles up to the one where the run ends, JG of them side by side.
constexpr int JG = 8;
__global__ void __launch_bounds__(32 * JG) combine_kernel(RedArgs a) {
  __shared__ float part[JG][32];
  const int lane = threadIdx.x & 31, jg = threadIdx.x >> 5;
  const long long pe = ((long long)blockIdx.x + 1) * a.R;   // first place behind the tile
  const uint32_t kk = a.keys[pe - 1];
  if (a.keys[pe] != kk || kk >= (uint32_t)a.V) return;
  const long long p0 = pe - a.R;
  if (p0 > 0 && a.keys[p0 - 1] == kk) return;               // it started before this tile
  long long lo = pe, hi = a.N;                              // first place behind the run
  while (lo < hi) {
    const long long mid = lo + ((hi - lo) >> 1);
    if (a.keys[mid] <= kk) lo = mid + 1;
    else hi = mid;
  }
  const int tl = (int)((lo - 1) / a.R);                     // the run's last tile
  for (int c0 = blockIdx.y * 32; c0 < a.D; c0 += gridDim.y * 32) {
    const int col = c0 + lane;
    float s = 0.f;
    if (col < a.D) {
      if (jg == 0) s = a.tail[(size_t)blockIdx.x * a.D + col];
#pragma unroll 8
      for (int q = (int)blockIdx.x + 1 + jg; q <= tl; q += JG) s += a.head[(size_t)q * a.D + col];
    }
    part[jg][lane] = s;
    __syncthreads();
    if (jg == 0 && col < a.D) {
      float acc = part[0][lane];
#pragma unroll
      for (int j = 1; j < JG; ++j) acc += part[j][lane];
      float one[1] = {acc};
      write_sum<1>(a, kk, col, one);
    }
    __syncthreads();
  }
}

template <typename T, int VE>
static e2f_status launch_reduce(RedArgs a, const T *g, cudaStream_t s) {
  const int dv = (a.D + VE - 1) / VE;
  const int RG = NT / a.CL;
  const size_t smem = sizeof(int) * (size_t)(2 * a.R + 2 + 2 * NT * VE + RG);
  const int zero = a.accumulate ? 0 : (a.V + ZROWS - 1) / ZROWS;
  dim3 grid((unsigned)(a.tiles + zero), (unsigned)((dv + a.CL - 1) / a.CL));
  E2F_LAUNCH((reduce_kernel<T, VE>), grid, NT, smem, s, a, g);
  if (a.tiles > 1) {
    dim3 cg((unsigned)(a.tiles - 1), (unsigned)std::min(64, (a.D + 31) / 32));
    E2F_LAUNCH(combine_kernel, cg, 32 * JG, 0, s, a);
  }
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
  const int dv = (D + VE - 1) / VE;
  a.CL = 1;
  while (a.CL < 32 && a.CL < dv) a.CL <<= 1;
  a.R = std::min(1024, 32 * (NT / a.CL));
  a.tiles = (N + a.R - 1) / a.R;
  SortArgs sa{};
  sa.N = N; sa.V = (int)V;
  const int subs = (N + SUB - 1) / SUB, per = (subs + MAX_TILES - 1) / MAX_TILES;
  sa.tile = per * SUB;
  const int st = (N + sa.tile - 1) / sa.tile;
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
  // keys run over 0 .. V (V: rows that take no part)
  E2F_LAUNCH((hist_kernel<I, true>), st, NT, 0, s, sa, ids, nullptr, hist, err);
  E2F_LAUNCH((scatter_kernel<I, true>), st, NT, 0, s, sa, ids, nullptr, nullptr, hist, k0, q0);
  for (sa.shift = 8; sa.shift < 32 && ((uint64_t)V >> sa.shift) != 0; sa.shift += 8) {
    E2F_LAUNCH((hist_kernel<I, false>), st, NT, 0, s, sa, nullptr, k0, hist, err);
    E2F_LAUNCH((scatter_kernel<I, false>), st, NT, 0, s, sa, nullptr, k0, q0, hist, k1, q1);
    std::swap(k0, k1);
    std::swap(q0, q1);
  }
  a.keys = k0;
  a.rows = q0;
  if (VE == W) return launch_reduce<T, W>(a, g, s);
  if (VE == 2) return launch_reduce<T, 2>(a, g, s);
  return launch_reduce<T, 1>(a, g, s);
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
