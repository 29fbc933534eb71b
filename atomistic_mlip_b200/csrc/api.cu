// C ABI of libe2f (declared in include/e2f.h): argument validation,
// dispatch to the kernels, the library's memory pool, diagnostics.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <vector>

#include "common.cuh"
#include "wigner.cuh"

namespace e2f {

std::atomic<int64_t> g_launches{0};
static thread_local char t_last_err[256] = "no CUDA error";

void set_cuda_error(cudaError_t e, const char *where) {
  snprintf(t_last_err, sizeof(t_last_err), "%s: %s", where, cudaGetErrorString(e));
}

// ---- per-device state: memory pool and error flag ---------------------------
// One slot per device in a fixed array: a pointer to a slot stays valid for
// the life of the process, whatever device another thread initialises.  The
// error flag is per device, shared by every stream of that device (see
// e2f_stream_status).
constexpr int MAX_DEVICES = 64;
struct DeviceState {
  cudaMemPool_t pool = nullptr;
  int *err_flag = nullptr;
};
static std::mutex g_mu;
static DeviceState g_dev[MAX_DEVICES];

// While it lives, this thread may allocate although a stream is being captured (what
// it allocates is not part of the captured work).
struct OutsideCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// An int of zero on the current device.
static int *new_flag() {
  int *p = nullptr;
  cudaStream_t s = nullptr;   // (the default stream may wait for a captured one)
  bool ok = cudaMalloc(&p, sizeof(int)) == cudaSuccess;
  ok = ok && cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess;
  ok = ok && cudaMemsetAsync(p, 0, sizeof(int), s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
  if (s) cudaStreamDestroy(s);
  if (!ok && p) cudaFree(p);
  return ok ? p : nullptr;
}

static DeviceState *device_state() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= MAX_DEVICES) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState &d = g_dev[dev];
  if (d.pool && d.err_flag) return &d;
  const OutsideCapture relaxed;   // the first call may be a captured one
  if (!d.pool) {
    cudaMemPoolProps props;
    memset(&props, 0, sizeof(props));
    props.allocType = cudaMemAllocationTypePinned;
    props.handleTypes = cudaMemHandleTypeNone;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    if (cudaMemPoolCreate(&d.pool, &props) != cudaSuccess) { d.pool = nullptr; return nullptr; }
    uint64_t thr = UINT64_MAX;   // keep freed blocks for reuse by later calls
    cudaMemPoolSetAttribute(d.pool, cudaMemPoolAttrReleaseThreshold, &thr);
  }
  if (!d.err_flag) d.err_flag = new_flag();
  return d.err_flag ? &d : nullptr;
}

cudaError_t pool_alloc(void **p, size_t bytes, cudaStream_t s) {
  DeviceState *d = device_state();
  if (!d) return cudaErrorInitializationError;
  return cudaMallocFromPoolAsync(p, bytes, d->pool, s);
}

int *device_error_flag() {
  DeviceState *d = device_state();
  return d ? d->err_flag : nullptr;
}

// ---- profiling of the dominant kernel ------------------------------------------
static std::atomic<bool> g_prof_on{false};
static std::mutex g_prof_mu;
static std::vector<std::pair<cudaEvent_t, cudaEvent_t>> g_prof_events;

static void prof_events(cudaEvent_t *a, cudaEvent_t *b) {
  *a = *b = nullptr;
  if (!g_prof_on.load()) return;
  if (cudaEventCreate(a) != cudaSuccess || cudaEventCreate(b) != cudaSuccess) { *a = *b = nullptr; return; }
  std::lock_guard<std::mutex> lk(g_prof_mu);
  g_prof_events.emplace_back(*a, *b);
}

// kernels (other translation units)
e2f_status build_neighbors_impl(const float *, int64_t, const float *, float, int32_t *, int32_t *, int64_t,
                                int64_t *, cudaStream_t);
e2f_status project_impl(const void *, int64_t, const e2f_weights *, void *, void *, void *, cudaStream_t);
template <typename T>
e2f_status attention_simt_impl(const T *, const T *, const T *, const float *, const e2f_csr *,
                               const e2f_weights *, float *, cudaStream_t, cudaEvent_t, cudaEvent_t);
e2f_status attention_tc_available(const e2f_weights *w);
e2f_status attention_tc_impl(const void *q, const void *k, const void *v, const float *pos, const e2f_csr *csr,
                             const e2f_weights *w, float *out, cudaStream_t s, cudaEvent_t ev0, cudaEvent_t ev1,
                             int F, const float *focus_a);

__global__ void wigner_kernel(const float *__restrict__ R, int64_t n, int L, float *__restrict__ D) {
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= n) return;
  float Rl[9];
  for (int k = 0; k < 9; ++k) Rl[k] = R[e * 9 + k];
  wig_all_serial(Rl, L, D + e * wig_size(L));
}

// Feature rows and weight matrices are read and written as 16-byte vectors.
static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static e2f_status validate_weights(const e2f_weights *w) {
  if (!w) return E2F_ERR_INVALID_ARG;
  if (w->L_max < 0 || w->L_max > E2F_MAX_L || w->C < 1 || w->H < 1) return E2F_ERR_INVALID_ARG;
  if (w->C % w->H != 0) return E2F_ERR_UNSUPPORTED;
  if (w->dtype != E2F_F32 && w->dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
  for (int l = 0; l <= w->L_max; ++l)
    if (!w->Wq[l] || !w->Wk[l] || !w->Wv[l]) return E2F_ERR_INVALID_ARG;
  if (!w->W0 || !w->rad_W1 || !w->rad_W2) return E2F_ERR_INVALID_ARG;
  for (int m = 1; m <= w->L_max; ++m)
    if (!w->Wr[m] || !w->Wi[m]) return E2F_ERR_INVALID_ARG;
  for (int l = 0; l <= w->L_max; ++l)
    if (!aligned16(w->Wq[l]) || !aligned16(w->Wk[l]) || !aligned16(w->Wv[l])) return E2F_ERR_INVALID_ARG;
  if (!aligned16(w->W0)) return E2F_ERR_INVALID_ARG;
  for (int m = 1; m <= w->L_max; ++m)
    if (!aligned16(w->Wr[m]) || !aligned16(w->Wi[m])) return E2F_ERR_INVALID_ARG;
  return E2F_OK;
}

static e2f_status validate_csr(const e2f_csr *csr) {
  if (!csr || csr->n_nodes < 0 || csr->n_edges < 0 || !(csr->r_c > 0.f)) return E2F_ERR_INVALID_ARG;
  if (csr->n_nodes > 0 && (!csr->row_ptr || (csr->n_edges > 0 && !csr->col_idx))) return E2F_ERR_INVALID_ARG;
  for (int k = 0; k < 3; ++k)
    if (csr->box[k] > 0.f && !(csr->r_c < 0.5f * csr->box[k])) return E2F_ERR_CUTOFF_TOO_LARGE;
  return E2F_OK;
}

e2f_status block_forward_impl(const float *x, const float *pos, const e2f_csr *csr, const e2f_block_weights *w,
                              float *out, cudaStream_t s);
int64_t cg_num_paths(int L);
e2f_status cg_conv_impl(const void *x, int dtype, const float *pos, const e2f_csr *csr, int L, int C,
                        const float *W, float *out, cudaStream_t s);
e2f_status attention_backward_impl(const void *x, const float *pos, const e2f_csr *csr, const e2f_weights *w,
                                   const float *G, float *dx, float *dpos, cudaStream_t s);

e2f_status embed_forward_impl(const void *ids, int id_type, int64_t N, const void *table, int dtype, int64_t V, int D,
                              float scale, int Q, void *out, int out_dtype, cudaStream_t s);
e2f_status embed_backward_impl(const void *ids, int id_type, int64_t N, const void *grad_out, int dtype, int64_t V, int D,
                               float scale, int Q, float *grad_table, int accumulate, cudaStream_t s);

e2f_status linear_forward_impl(const e2f_linear *p, const void *residual, int64_t ldr, void *out, int64_t ldo,
                               int out_dtype, cudaStream_t s);
e2f_status linear_backward_impl(const e2f_linear *p, const void *grad_out, int64_t ldg, int out_dtype, void *grad_x,
                                int64_t ldgx, void *grad_W, int64_t ldgw, float *grad_bias, cudaStream_t s);

static bool float_type(int32_t t) { return t == E2F_F32 || t == E2F_BF16; }
static bool aligned_elem(const void *p, int32_t type) {
  const uintptr_t b = type == E2F_BF16 ? 2 : type == E2F_I64 ? 8 : 4;
  return reinterpret_cast<uintptr_t>(p) % b == 0;
}

static e2f_status validate_embed(int32_t id_type, int64_t N, int32_t dtype, int64_t V, int32_t D, float scale, int32_t Q) {
  if (id_type != E2F_I32 && id_type != E2F_I64) return E2F_ERR_UNSUPPORTED;
  if (!float_type(dtype)) return E2F_ERR_UNSUPPORTED;
  if (N < 0 || N > E2F_MAX_ROWS || V < 1 || V > E2F_MAX_ROWS || D < 1 || Q < 1) return E2F_ERR_INVALID_ARG;
  if (D > (1 << 20) || (int64_t)Q * D > (1 << 30)) return E2F_ERR_UNSUPPORTED;
  if (!(scale > -INFINITY && scale < INFINITY)) return E2F_ERR_INVALID_ARG;
  return E2F_OK;
}

// A row stride in elements: wide enough, and small enough that the byte offset of any row fits 62 bits.
static bool stride_ok(int64_t ld, int32_t cols) { return ld >= cols && ld <= ((int64_t)1 << 29); }

static e2f_status validate_linear(const e2f_linear *p, int32_t out_dtype) {
  if (!p) return E2F_ERR_INVALID_ARG;
  if (!float_type(p->dtype) || !float_type(out_dtype)) return E2F_ERR_UNSUPPORTED;
  if (p->act != E2F_ACT_NONE && p->act != E2F_ACT_SILU && p->act != E2F_ACT_GELU) return E2F_ERR_UNSUPPORTED;
  if (p->M < 0 || p->M > E2F_MAX_ROWS || p->K < 1 || p->N < 1) return E2F_ERR_INVALID_ARG;
  if (p->K > (1 << 20) || p->N > (1 << 20)) return E2F_ERR_UNSUPPORTED;
  if (!stride_ok(p->ldx, p->K) || !stride_ok(p->ldw, p->K)) return E2F_ERR_INVALID_ARG;
  if (p->M > 0 && (!p->x || !p->W)) return E2F_ERR_INVALID_ARG;
  if (!aligned_elem(p->x, p->dtype) || !aligned_elem(p->W, p->dtype) || !aligned_elem(p->bias, E2F_F32))
    return E2F_ERR_INVALID_ARG;
  return E2F_OK;
}

// q, k, v (library scratch), then the fused attention kernel; arguments
// already validated.
e2f_status attention_forward_impl(const void *x, const float *pos, const e2f_csr *csr, const e2f_weights *w,
                                  float *out, cudaStream_t s, int F = 1, const float *focus_a = nullptr) {
  const int64_t N = csr->n_nodes;
  if (N == 0) return E2F_OK;
  const size_t Q = (size_t)(w->L_max + 1) * (w->L_max + 1);
  const size_t esz = w->dtype == E2F_F32 ? 4 : 2;
  const size_t feat = (size_t)N * Q * w->C * esz;
  Scratch qkv;
  E2F_CUDA_TRY(qkv.alloc(3 * feat, s));
  char *base = qkv.as<char>();
  void *q = base, *k = base + feat, *v = base + 2 * feat;
  e2f_status st = project_impl(x, N, w, q, k, v, s);
  if (st != E2F_OK) return st;
  cudaEvent_t ev0, ev1;
  prof_events(&ev0, &ev1);
  if (F > 1) {   // multi-focus: the tensor-core kernel only (checked by the caller)
    return attention_tc_impl(q, k, v, pos, csr, w, out, s, ev0, ev1, F, focus_a);
  }
  if (w->dtype == E2F_BF16 && attention_tc_available(w) == E2F_OK)
    return attention_tc_impl(q, k, v, pos, csr, w, out, s, ev0, ev1, 1, nullptr);
  if (w->dtype == E2F_F32)
    return attention_simt_impl<float>((const float *)q, (const float *)k, (const float *)v, pos, csr, w, out, s,
                                      ev0, ev1);
  return attention_simt_impl<__nv_bfloat16>((const __nv_bfloat16 *)q, (const __nv_bfloat16 *)k,
                                            (const __nv_bfloat16 *)v, pos, csr, w, out, s, ev0, ev1);
}

}  // namespace e2f

using namespace e2f;

extern "C" {

const char *e2f_status_string(e2f_status s) {
  switch (s) {
    case E2F_OK: return "ok";
    case E2F_ERR_INVALID_ARG: return "invalid argument";
    case E2F_ERR_CUTOFF_TOO_LARGE: return "cutoff >= half the periodic box";
    case E2F_ERR_CAPACITY: return "col_idx capacity too small";
    case E2F_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case E2F_ERR_CUDA: return "CUDA error";
    case E2F_ERR_TIMEOUT: return "bounded device wait timed out";
    case E2F_ERR_DOMAIN: return "coordinate outside the periodic box";
    case E2F_ERR_SCRATCH_LIMIT: return "input exceeds the fixed scratch of a no-allocation entry point";
    default: return "unknown status";
  }
}

const char *e2f_last_cuda_error(void) { return t_last_err; }

e2f_status e2f_build_neighbors(const float *pos, int64_t N, const float *box, float r_c, int32_t *row_ptr,
                               int32_t *col_idx, int64_t capacity, int64_t *n_edges, e2f_csr *out_csr,
                               void *stream) {
  if (N < 0 || N > INT32_MAX - 1 || !n_edges || !row_ptr || capacity < 0) return E2F_ERR_INVALID_ARG;
  if (N > 0 && !pos) return E2F_ERR_INVALID_ARG;
  if (capacity > 0 && !col_idx) return E2F_ERR_INVALID_ARG;
  if (!(r_c > 0.f) || !(r_c < INFINITY)) return E2F_ERR_INVALID_ARG;
  if (box) {
    for (int k = 0; k < 3; ++k) {
      if (!(box[k] >= 0.f) || !(box[k] < INFINITY)) return E2F_ERR_INVALID_ARG;
      if (box[k] > 0.f && !(r_c < 0.5f * box[k])) return E2F_ERR_CUTOFF_TOO_LARGE;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e2f_status st = build_neighbors_impl(pos, N, box, r_c, row_ptr, col_idx, capacity, n_edges, s);
  if (st != E2F_OK && st != E2F_ERR_CAPACITY) return st;
  if (out_csr) {
    out_csr->row_ptr = row_ptr;
    out_csr->col_idx = col_idx;
    out_csr->n_nodes = N;
    out_csr->n_edges = *n_edges;
    for (int k = 0; k < 3; ++k) out_csr->box[k] = box ? box[k] : 0.f;
    out_csr->r_c = r_c;
  }
  return st;
}

e2f_status e2f_project_qkv(const void *x, int64_t N, const e2f_weights *w, void *q, void *k, void *v,
                           void *stream) {
  e2f_status st = validate_weights(w);
  if (st != E2F_OK) return st;
  if (N < 0) return E2F_ERR_INVALID_ARG;
  if (N > 0 && (!x || !q || !k || !v)) return E2F_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(k) || !aligned16(v)) return E2F_ERR_INVALID_ARG;
  return project_impl(x, N, w, q, k, v, static_cast<cudaStream_t>(stream));
}

e2f_status e2f_attention_forward(const void *x, const float *pos, const e2f_csr *csr, const e2f_weights *w,
                                 float *out, void *stream) {
  e2f_status st = validate_weights(w);
  if (st != E2F_OK) return st;
  st = validate_csr(csr);
  if (st != E2F_OK) return st;
  if (csr->n_nodes == 0) return E2F_OK;
  if (!x || !pos || !out) return E2F_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(out)) return E2F_ERR_INVALID_ARG;
  return attention_forward_impl(x, pos, csr, w, out, static_cast<cudaStream_t>(stream));
}

e2f_status e2f_attention_backward(const void *x, const float *pos, const e2f_csr *csr, const e2f_weights *w,
                                  const float *grad_out, float *grad_x, float *grad_pos, void *stream) {
  e2f_status st = validate_weights(w);
  if (st != E2F_OK) return st;
  st = validate_csr(csr);
  if (st != E2F_OK) return st;
  if (w->H > 16) return E2F_ERR_UNSUPPORTED;
  if (csr->n_nodes == 0) return E2F_OK;
  if (!x || !pos || !grad_out || !grad_x || !grad_pos) return E2F_ERR_INVALID_ARG;
  if (!aligned16(x)) return E2F_ERR_INVALID_ARG;
  return attention_backward_impl(x, pos, csr, w, grad_out, grad_x, grad_pos, static_cast<cudaStream_t>(stream));
}

e2f_status e2f_block_forward(const float *x, const float *pos, const e2f_csr *csr, const e2f_block_weights *w,
                             float *out, void *stream) {
  if (!w) return E2F_ERR_INVALID_ARG;
  e2f_status st = validate_weights(&w->attn);
  if (st != E2F_OK) return st;
  st = validate_csr(csr);
  if (st != E2F_OK) return st;
  const int L = w->attn.L_max;
  if (w->hidden < 1 || !w->gamma1 || !w->gamma2 || !w->Wa || !aligned16(w->Wa)) return E2F_ERR_INVALID_ARG;
  for (int l = 0; l <= L; ++l)
    if (!w->Wb[l] || !w->Wd[l] || !aligned16(w->Wb[l]) || !aligned16(w->Wd[l])) return E2F_ERR_INVALID_ARG;
  if (csr->n_nodes == 0) return E2F_OK;
  if (!x || !pos || !out || x == out) return E2F_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(out)) return E2F_ERR_INVALID_ARG;
  return block_forward_impl(x, pos, csr, w, out, static_cast<cudaStream_t>(stream));
}

e2f_status e2f_attention_forward_multifocus(const void *x, const float *pos, const e2f_csr *csr, const e2f_weights *w,
                                            int32_t F, const float *focus_a, float *out, void *stream) {
  e2f_status st = validate_weights(w);
  if (st != E2F_OK) return st;
  st = validate_csr(csr);
  if (st != E2F_OK) return st;
  if (F != 1 && F != 2 && F != 4 && F != 8) return E2F_ERR_INVALID_ARG;
  if (F > 1) {
    if (attention_tc_available(w) != E2F_OK || (w->L_max != 2 && w->L_max != 4)) return E2F_ERR_UNSUPPORTED;
    if (!focus_a || !aligned16(focus_a)) return E2F_ERR_INVALID_ARG;
  }
  if (csr->n_nodes == 0) return E2F_OK;
  if (!x || !pos || !out) return E2F_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(out)) return E2F_ERR_INVALID_ARG;
  return attention_forward_impl(x, pos, csr, w, out, static_cast<cudaStream_t>(stream), F, focus_a);
}

int64_t e2f_cg_num_paths(int32_t L) {
  if (L < 0 || L > E2F_MAX_L) return -1;
  return cg_num_paths(L);
}

e2f_status e2f_cg_conv_forward(const void *x, int32_t dtype, const float *pos, const e2f_csr *csr, int32_t L,
                               int32_t C, const float *W, float *out, void *stream) {
  e2f_status st = validate_csr(csr);
  if (st != E2F_OK) return st;
  if (L < 0 || L > E2F_MAX_L) return E2F_ERR_UNSUPPORTED;
  if (dtype != E2F_F32 && dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
  if (C < 2 || C > 256 || (C & 1)) return E2F_ERR_INVALID_ARG;
  if (csr->n_nodes == 0) return E2F_OK;
  if (!x || !pos || !W || !out) return E2F_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(out)) return E2F_ERR_INVALID_ARG;
  return cg_conv_impl(x, dtype, pos, csr, L, C, W, out, static_cast<cudaStream_t>(stream));
}

e2f_status e2f_embed_forward(const void *ids, int32_t id_type, int64_t N, const void *table, int32_t dtype, int64_t V,
                             int32_t D, float scale, int32_t Q, void *out, int32_t out_dtype, void *stream) {
  e2f_status st = validate_embed(id_type, N, dtype, V, D, scale, Q);
  if (st != E2F_OK) return st;
  if (!float_type(out_dtype)) return E2F_ERR_UNSUPPORTED;
  if (N == 0) return E2F_OK;
  if (!ids || !table || !out || out == table || out == ids) return E2F_ERR_INVALID_ARG;
  if (!aligned_elem(ids, id_type) || !aligned_elem(table, dtype) || !aligned_elem(out, out_dtype))
    return E2F_ERR_INVALID_ARG;
  return embed_forward_impl(ids, id_type, N, table, dtype, V, D, scale, Q, out, out_dtype,
                            static_cast<cudaStream_t>(stream));
}

e2f_status e2f_embed_backward(const void *ids, int32_t id_type, int64_t N, const void *grad_out, int32_t dtype, int64_t V,
                              int32_t D, float scale, int32_t Q, float *grad_table, int32_t accumulate, void *stream) {
  e2f_status st = validate_embed(id_type, N, dtype, V, D, scale, Q);
  if (st != E2F_OK) return st;
  if (accumulate != 0 && accumulate != 1) return E2F_ERR_INVALID_ARG;
  if (!grad_table || !aligned_elem(grad_table, E2F_F32)) return E2F_ERR_INVALID_ARG;
  if (N > 0 && (!ids || !grad_out || grad_table == grad_out || grad_table == ids)) return E2F_ERR_INVALID_ARG;
  if (!aligned_elem(ids, id_type) || !aligned_elem(grad_out, dtype)) return E2F_ERR_INVALID_ARG;
  return embed_backward_impl(ids, id_type, N, grad_out, dtype, V, D, scale, Q, grad_table, accumulate,
                             static_cast<cudaStream_t>(stream));
}

e2f_status e2f_linear_forward(const e2f_linear *p, const void *residual, int64_t ldr, void *out, int64_t ldo,
                              int32_t out_dtype, void *stream) {
  e2f_status st = validate_linear(p, out_dtype);
  if (st != E2F_OK) return st;
  if (!stride_ok(ldo, p->N) || (residual && !stride_ok(ldr, p->N))) return E2F_ERR_INVALID_ARG;
  if (p->M == 0) return E2F_OK;
  if (!out || out == p->x || out == p->W || out == p->bias) return E2F_ERR_INVALID_ARG;
  if (residual == out && ldr != ldo) return E2F_ERR_INVALID_ARG;
  if (!aligned_elem(out, out_dtype) || !aligned_elem(residual, out_dtype)) return E2F_ERR_INVALID_ARG;
  return linear_forward_impl(p, residual, ldr, out, ldo, out_dtype, static_cast<cudaStream_t>(stream));
}

e2f_status e2f_linear_backward(const e2f_linear *p, const void *grad_out, int64_t ldg, int32_t out_dtype, void *grad_x,
                               int64_t ldgx, void *grad_W, int64_t ldgw, float *grad_bias, void *stream) {
  e2f_status st = validate_linear(p, out_dtype);
  if (st != E2F_OK) return st;
  if (!stride_ok(ldg, p->N) || (grad_x && !stride_ok(ldgx, p->K)) || (grad_W && !stride_ok(ldgw, p->K)))
    return E2F_ERR_INVALID_ARG;
  if (p->M > 0 && !grad_out) return E2F_ERR_INVALID_ARG;
  for (const void *o : {(const void *)grad_x, (const void *)grad_W, (const void *)grad_bias})
    if (o && (o == p->x || o == p->W || o == p->bias || o == grad_out)) return E2F_ERR_INVALID_ARG;
  if ((grad_x && (grad_x == grad_W || grad_x == grad_bias)) || (grad_W && grad_W == grad_bias)) return E2F_ERR_INVALID_ARG;
  if (!aligned_elem(grad_out, out_dtype) || !aligned_elem(grad_x, p->dtype) || !aligned_elem(grad_W, p->dtype) ||
      !aligned_elem(grad_bias, E2F_F32))
    return E2F_ERR_INVALID_ARG;
  return linear_backward_impl(p, grad_out, ldg, out_dtype, grad_x, ldgx, grad_W, ldgw, grad_bias,
                              static_cast<cudaStream_t>(stream));
}

e2f_status e2f_stream_status(void *stream) {
  E2F_CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  int *flag = device_error_flag();
  if (!flag) return E2F_ERR_CUDA;
  int h = 0;
  E2F_CUDA_TRY(cudaMemcpy(&h, flag, sizeof(int), cudaMemcpyDeviceToHost));
  if (h) {
    E2F_CUDA_TRY(cudaMemset(flag, 0, sizeof(int)));
    return h;
  }
  return E2F_OK;
}

e2f_status e2f_wigner_d(const float *R, int64_t n, int32_t L, float *D, void *stream) {
  if (n < 0 || L < 0 || L > E2F_MAX_L) return E2F_ERR_INVALID_ARG;
  if (n == 0) return E2F_OK;
  if (!R || !D) return E2F_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  E2F_LAUNCH(wigner_kernel, (unsigned)((n + 127) / 128), 128, 0, s, R, n, L, D);
  return E2F_OK;
}

int64_t e2f_kernel_launches(void) { return g_launches.load(); }

e2f_status e2f_profile_enable(int32_t on) {
  g_prof_on = on != 0;
  return E2F_OK;
}

e2f_status e2f_profile_read(int64_t *launches, double *total_ms) {
  if (!launches || !total_ms) return E2F_ERR_INVALID_ARG;
  double tot = 0.0;
  int64_t n = 0;
  e2f_status st = E2F_OK;
  std::lock_guard<std::mutex> lk(g_prof_mu);
  for (auto &pr : g_prof_events) {
    float ms = 0.f;
    if (cudaEventSynchronize(pr.second) != cudaSuccess || cudaEventElapsedTime(&ms, pr.first, pr.second) != cudaSuccess)
      st = E2F_ERR_CUDA;
    tot += ms;
    ++n;
    cudaEventDestroy(pr.first);
    cudaEventDestroy(pr.second);
  }
  g_prof_events.clear();
  *launches = n;
  *total_ms = tot;
  return st;
}

e2f_status e2f_scratch_high_water(int64_t *bytes, int32_t reset) {
  if (!bytes) return E2F_ERR_INVALID_ARG;
  DeviceState *d = device_state();
  if (!d) return E2F_ERR_CUDA;
  uint64_t v = 0;
  E2F_CUDA_TRY(cudaMemPoolGetAttribute(d->pool, cudaMemPoolAttrUsedMemHigh, &v));
  *bytes = (int64_t)v;
  if (reset) {
    uint64_t z = 0;
    E2F_CUDA_TRY(cudaMemPoolSetAttribute(d->pool, cudaMemPoolAttrUsedMemHigh, &z));
  }
  return E2F_OK;
}

}  // extern "C"
