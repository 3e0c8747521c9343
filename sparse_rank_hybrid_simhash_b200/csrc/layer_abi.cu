// The C ABI of the operators next to ELSAA: validation, workspace layout and
// launches of the norm and rotation, the window attention and the paged cache
// (see include/elsaa.h).
#include <limits.h>
#include <math.h>

#include "internal.h"
#include "layer.h"
#include "paged_runs.cuh"

using namespace elsaa;

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }

bool head_dim(int d, elsaa_status* why) {
  if (d <= 0) return false;
  if (d != 32 && d != 64 && d != 128) {
    *why = ELSAA_ERR_UNSUPPORTED;
    return false;
  }
  return true;
}

bool shape_ok(int B, int H, int Hkv, int N, int d, int dtype, elsaa_status* why) {
  *why = ELSAA_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || Hkv <= 0 || N <= 0 || H > 16384 || H % Hkv != 0) return false;
  if (dtype != ELSAA_BF16 && dtype != ELSAA_F32) return false;
  // rows are numbered in 32 bits, with room for the last tile (elements and bytes in 64)
  if ((int64_t)B * H > INT32_MAX || (int64_t)B * H * N > INT32_MAX - 4096) return false;
  return head_dim(d, why);
}

elsaa_status check(const elsaa_rotary_params* p) {
  elsaa_status why = ELSAA_ERR_INVALID_ARG;
  if (!p || !shape_ok(p->B, p->H, p->Hkv, p->N, p->d, p->dtype, &why)) return why;
  if (p->rot_dim < 0 || p->rot_dim > p->d || p->rot_dim % 16 != 0) return ELSAA_ERR_INVALID_ARG;
  if ((p->interleaved != 0 && p->interleaved != 1) || (p->norm != 0 && p->norm != 1))
    return ELSAA_ERR_INVALID_ARG;
  if (p->rot_dim > 0 && p->max_pos <= 0) return ELSAA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || isinf(p->eps)) return ELSAA_ERR_INVALID_ARG;
  return ELSAA_OK;
}

elsaa_status check(const elsaa_window_params* p) {
  elsaa_status why = ELSAA_ERR_INVALID_ARG;
  if (!p || !shape_ok(p->B, p->H, p->Hkv, p->N, p->d, p->dtype, &why)) return why;
  if (p->window < 0 || p->sinks < 0 || isnan(p->scale) || isinf(p->scale))
    return ELSAA_ERR_INVALID_ARG;
  // (the rows padded to whole tiles, too)
  if ((int64_t)p->B * p->H * (((int64_t)p->N + 127) / 128 * 128) > INT32_MAX - 4096)
    return ELSAA_ERR_INVALID_ARG;
  return ELSAA_OK;
}

elsaa_status check(const elsaa_paged_params* p) {
  elsaa_status why = ELSAA_ERR_INVALID_ARG;
  if (!p || !shape_ok(1, p->H, p->Hkv, p->rows, p->d, p->dtype, &why)) return why;
  if (p->seqs <= 0 || p->pages <= 0 || p->table_width <= 0) return ELSAA_ERR_INVALID_ARG;
  if (p->page_size <= 0 || p->page_size % 16 != 0) return ELSAA_ERR_INVALID_ARG;
  if (p->window < 0 || p->sinks < 0 || isnan(p->scale) || isinf(p->scale))
    return ELSAA_ERR_INVALID_ARG;
  // positions are 32-bit, with room for a block behind the last one
  if ((int64_t)p->page_size * p->table_width > INT32_MAX - 1024) return ELSAA_ERR_INVALID_ARG;
  if ((int64_t)p->seqs * p->table_width > INT32_MAX) return ELSAA_ERR_INVALID_ARG;
  if (p->H / p->Hkv > 64) return ELSAA_ERR_UNSUPPORTED;
  return ELSAA_OK;
}

// Strides of a tensor of the given extents: the caller's, or dense.  Sizes of
// one do not move, so their stride is replaced by the dense one.
bool take_strides(const int64_t* given, int64_t b, int64_t h, int64_t n, int64_t d, int esz,
                  Strides* out) {
  const Strides dense{h * n * d, n * d, d};
  *out = dense;
  if (!given) return true;
  const int64_t size[3] = {b, h, n};
  int64_t* to[3] = {&out->b, &out->h, &out->n};
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    const int64_t x = given[i];
    // (a tensor map holds strides below 2^40 bytes)
    if (x < d || (x * esz) % 16 != 0 || x >= ((int64_t)1 << 40) / esz) return false;
    *to[i] = x;
  }
  return true;
}

// (row, head) strides of a [T, heads, d] tensor, as one batch.
bool take_row_strides(const int64_t* given, int64_t rows, int64_t h, int64_t d, int esz,
                      Strides* out) {
  const int64_t x[3] = {rows * h * d, given ? given[1] : d, given ? given[0] : h * d};
  return take_strides(x, 1, h, rows, d, esz, out);
}

// Whether one of the `outs` last of n tensors starts where another tensor does.  (Views of one
// buffer may lie inside one another's range without sharing an element, so that is all that is
// refused of what the contract rules out.)
bool shared_start(const void* const* t, int n, int outs) {
  for (int o = n - outs; o < n; ++o)
    for (int i = 0; i < o; ++i)
      if (t[i] == t[o]) return true;
  return false;
}

inline int esize(int dtype) { return dtype == ELSAA_BF16 ? 2 : 4; }

elsaa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ELSAA_OK : ELSAA_ERR_CUDA; }

}  // namespace

extern "C" {

// ---- norm and rotation -------------------------------------------------------

elsaa_status elsaa_rotary_validate(const elsaa_rotary_params* p) { return check(p); }

size_t elsaa_rotary_workspace_bytes(const elsaa_rotary_params* p) {
  if (check(p) != ELSAA_OK) return 0;
  return kHeadBytes + (size_t)kRotaryPartials * p->d * sizeof(float);
}

static elsaa_status rotary_args(const elsaa_rotary_params* p, const float* table, const float* wq,
                                const float* wk, void* ws, size_t ws_bytes, RotaryArgs* a) {
  const elsaa_status st = check(p);
  if (st != ELSAA_OK) return st;
  if (!ws || ((uintptr_t)ws & 255) != 0 || (p->rot_dim > 0 && !table)) return ELSAA_ERR_INVALID_ARG;
  if (!aligned16(table) || !aligned16(wq) || !aligned16(wk)) return ELSAA_ERR_INVALID_ARG;
  if (ws_bytes < elsaa_rotary_workspace_bytes(p)) return ELSAA_ERR_WORKSPACE;
  a->table = table;
  a->wq = p->norm ? wq : nullptr;
  a->wk = p->norm ? wk : nullptr;
  a->err = (uint32_t*)ws;
  a->partials = (float*)((char*)ws + kHeadBytes);
  a->B = p->B;
  a->H = p->H;
  a->Hkv = p->Hkv;
  a->N = p->N;
  a->rot = p->rot_dim;
  a->norm = p->norm;
  a->max_pos = p->max_pos;
  a->eps = p->eps;
  return ELSAA_OK;
}

// Without positions the tokens are 0 .. N - 1: the table has to hold them all (positions are
// known to the device alone, which records those outside).
static bool token_order_ok(const elsaa_rotary_params* p, const int32_t* positions) {
  return positions || p->rot_dim == 0 || p->N <= p->max_pos;
}

elsaa_status elsaa_rotary_forward(const elsaa_rotary_params* p, const void* q, const void* k,
                                  const int64_t* strides, const int32_t* positions,
                                  const float* table, const float* q_weight,
                                  const float* k_weight, void* qo, void* ko, void* ws,
                                  size_t ws_bytes, void* stream) {
  RotaryArgs a = {};
  const elsaa_status st = rotary_args(p, table, q_weight, k_weight, ws, ws_bytes, &a);
  if (st != ELSAA_OK) return st;
  if (!token_order_ok(p, positions)) return ELSAA_ERR_INVALID_ARG;
  if (!q || !qo || (k == nullptr) != (ko == nullptr) || !aligned4(positions)) return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {q, k, (const void*)qo, (const void*)ko})
    if (!aligned16(x)) return ELSAA_ERR_INVALID_ARG;
  const int e = esize(p->dtype);
  auto take = [&](int i, int h, Strides* to) {
    return take_strides(strides ? strides + 3 * i : nullptr, p->B, h, p->N, p->d, e, to);
  };
  if (!take(0, p->H, &a.sq) || !take(2, p->H, &a.sqo) ||
      (k && (!take(1, p->Hkv, &a.sk) || !take(3, p->Hkv, &a.sko))))
    return ELSAA_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.qo = qo;
  a.ko = ko;
  a.positions = positions;
  if (!k) a.Hkv = 0;
  return cuda_status(launch_rotary_forward(a, p->d, p->dtype == ELSAA_BF16, p->interleaved != 0,
                                           (cudaStream_t)stream));
}

elsaa_status elsaa_rotary_backward(const elsaa_rotary_params* p, const void* q, const void* k,
                                   const int64_t* strides, const int32_t* positions,
                                   const float* table, const float* q_weight,
                                   const float* k_weight, const void* dqo, const void* dko,
                                   void* dq, void* dk, float* dq_weight, float* dk_weight,
                                   void* ws, size_t ws_bytes, void* stream) {
  RotaryArgs a = {};
  const elsaa_status st = rotary_args(p, table, q_weight, k_weight, ws, ws_bytes, &a);
  if (st != ELSAA_OK) return st;
  if (!token_order_ok(p, positions)) return ELSAA_ERR_INVALID_ARG;
  if (!q || !dqo || !dq || (k == nullptr) != (dko == nullptr) || (k == nullptr) != (dk == nullptr))
    return ELSAA_ERR_INVALID_ARG;
  if (!p->norm && (dq_weight || dk_weight)) return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {(const void*)positions, (const void*)dq_weight, (const void*)dk_weight})
    if (!aligned4(x)) return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {q, k, dqo, dko, (const void*)dq, (const void*)dk})
    if (!aligned16(x)) return ELSAA_ERR_INVALID_ARG;
  const int e = esize(p->dtype);
  auto take = [&](int i, int h, Strides* to) {
    return take_strides(strides ? strides + 3 * i : nullptr, p->B, h, p->N, p->d, e, to);
  };
  if (!take(0, p->H, &a.sq) || !take(2, p->H, &a.sdqo) || !take(4, p->H, &a.sqo) ||
      (k && (!take(1, p->Hkv, &a.sk) || !take(3, p->Hkv, &a.sdko) || !take(5, p->Hkv, &a.sko))))
    return ELSAA_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.dqo = dqo;
  a.dko = dko;
  a.qo = dq;
  a.ko = dk;
  a.dwq = dq_weight;
  a.dwk = k ? dk_weight : nullptr;
  a.positions = positions;
  if (!k) a.Hkv = 0;
  return cuda_status(launch_rotary_backward(a, p->d, p->dtype == ELSAA_BF16, p->interleaved != 0,
                                            (cudaStream_t)stream));
}

// ---- window attention ----------------------------------------------------------

elsaa_status elsaa_window_validate(const elsaa_window_params* p) { return check(p); }

size_t elsaa_window_workspace_bytes(const elsaa_window_params* p, int32_t backward) {
  if (check(p) != ELSAA_OK) return 0;
  if (!backward) return kHeadBytes;
  return kHeadBytes + (attend_tc_supported(p->d, p->dtype == ELSAA_BF16)
                           ? window_tc_scratch_bytes(p->d, p->B, p->H, p->N)
                           : window_simt_scratch_bytes(p->d, p->B, p->H, p->Hkv, p->N,
                                                       p->window > 0 ? p->window : INT32_MAX, p->sinks));
}

static elsaa_status window_args(const elsaa_window_params* p, const void* const* tensors,
                                int count, const int64_t* strides, const int32_t* lengths,
                                void* ws, size_t ws_bytes, bool backward, AttendArgs* a) {
  const elsaa_status st = check(p);
  if (st != ELSAA_OK) return st;
  if (!ws || ((uintptr_t)ws & 255) != 0) return ELSAA_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (!tensors[i] || !aligned16(tensors[i])) return ELSAA_ERR_INVALID_ARG;
  if (ws_bytes < elsaa_window_workspace_bytes(p, backward ? 1 : 0)) return ELSAA_ERR_WORKSPACE;
  Strides* to[8] = {&a->sq, &a->sk, &a->sv, &a->sy, &a->sdy, &a->sdq, &a->sdk, &a->sdv};
  const bool kv[8] = {false, true, true, false, false, false, true, true};
  for (int i = 0; i < count; ++i)
    if (!take_strides(strides ? strides + 3 * i : nullptr, p->B, kv[i] ? p->Hkv : p->H, p->N, p->d,
                      esize(p->dtype), to[i]))
      return ELSAA_ERR_INVALID_ARG;
  a->q = tensors[0];
  a->k = tensors[1];
  a->v = tensors[2];
  a->y = const_cast<void*>(tensors[3]);
  a->lengths = lengths;
  a->B = p->B;
  a->H = p->H;
  a->Hkv = p->Hkv;
  a->N = p->N;
  a->d = p->d;
  a->g = p->H / p->Hkv;
  a->window = p->window > 0 ? p->window : INT32_MAX;
  a->sinks = p->sinks;
  a->scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->d);
  a->err = (uint32_t*)ws;
  a->counters = (uint32_t*)((char*)ws + kCounters);
  a->delta = (float*)((char*)ws + kHeadBytes);
  return ELSAA_OK;
}

elsaa_status elsaa_window_forward(const elsaa_window_params* p, const void* q, const void* k,
                                  const void* v, const int64_t* strides, const int32_t* lengths,
                                  void* y, float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttendArgs a = {};
  const void* t[4] = {q, k, v, y};
  const elsaa_status st = window_args(p, t, 4, strides, lengths, ws, ws_bytes, false, &a);
  if (st != ELSAA_OK) return st;
  if (!lse || !aligned4(lse) || !aligned4(lengths) || shared_start(t, 4, 1)) return ELSAA_ERR_INVALID_ARG;
  a.lse = lse;
  const bool bf16 = p->dtype == ELSAA_BF16;
  return cuda_status(attend_tc_supported(p->d, bf16)
                         ? launch_window_fwd_tc(a, (cudaStream_t)stream)
                         : launch_window_fwd_simt(a, bf16, (cudaStream_t)stream));
}

elsaa_status elsaa_window_backward(const elsaa_window_params* p, const void* q, const void* k,
                                   const void* v, const int64_t* strides, const int32_t* lengths,
                                   const void* y, const float* lse, const void* dy, void* dq,
                                   void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  AttendArgs a = {};
  const void* t[8] = {q, k, v, y, dy, dq, dk, dv};
  const elsaa_status st = window_args(p, t, 8, strides, lengths, ws, ws_bytes, true, &a);
  if (st != ELSAA_OK) return st;
  if (!lse || !aligned4(lse) || !aligned4(lengths) || shared_start(t, 8, 3)) return ELSAA_ERR_INVALID_ARG;
  a.lse = const_cast<float*>(lse);
  a.dy = dy;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  const bool bf16 = p->dtype == ELSAA_BF16;
  if (attend_tc_supported(p->d, bf16)) return cuda_status(launch_window_bwd_tc(a, (cudaStream_t)stream));
  cudaError_t e = launch_window_delta(a, bf16, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_window_bwd_simt(a, bf16, (cudaStream_t)stream);
  return cuda_status(e);
}

// ---- paged cache ---------------------------------------------------------------

elsaa_status elsaa_paged_validate(const elsaa_paged_params* p) { return check(p); }

size_t elsaa_paged_workspace_bytes(const elsaa_paged_params* p) {
  if (check(p) != ELSAA_OK) return 0;
  const bool bf16 = p->dtype == ELSAA_BF16;
  const int g = p->H / p->Hkv;
  // (the tensor-core kernel's, or the kernels' with 64-key blocks)
  if (attend_tc_supported(p->d, bf16) && !paged_decode_supported(p->d, bf16, p->rows, p->seqs, g))
    return kHeadBytes + paged_scratch_bytes(p->d, p->rows, g);
  return kHeadBytes + paged_runs_bytes(p->d, paged_tile_rows(p->rows, p->seqs, g));
}

static bool page_strides_of(const elsaa_paged_params* p, const int64_t* given, Strides* kp,
                            Strides* vp) {
  const int e = esize(p->dtype);
  return take_strides(given, p->pages, p->Hkv, p->page_size, p->d, e, kp) &&
         take_strides(given ? given + 3 : nullptr, p->pages, p->Hkv, p->page_size, p->d, e, vp);
}

elsaa_status elsaa_paged_write(const elsaa_paged_params* p, const elsaa_rotary_params* r,
                               const void* q, const void* k, const void* v,
                               const int64_t* strides, const float* table,
                               const float* q_weight, const float* k_weight, void* q_out,
                               void* k_pages, void* v_pages, const int64_t* page_strides,
                               const int32_t* page_table, const int32_t* starts,
                               const int32_t* lengths, void* ws, size_t ws_bytes, void* stream) {
  elsaa_status st = check(p);
  if (st != ELSAA_OK) return st;
  if (!r || r->H != p->H || r->Hkv != p->Hkv || r->d != p->d || r->dtype != p->dtype)
    return ELSAA_ERR_INVALID_ARG;
  elsaa_rotary_params rp = *r;
  rp.B = 1;
  rp.N = p->rows;
  RotaryArgs a = {};
  // no partial sums here: the error word is all of the workspace
  st = rotary_args(&rp, table, q_weight, k_weight, ws, elsaa_rotary_workspace_bytes(&rp), &a);
  if (st != ELSAA_OK) return st;
  if (!q || !k || !v || !q_out || !k_pages || !v_pages || !page_table || !starts || !lengths)
    return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, (const void*)q_out, (const void*)k_pages, (const void*)v_pages})
    if (!aligned16(x)) return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {page_table, starts, lengths})
    if (!aligned4(x)) return ELSAA_ERR_INVALID_ARG;
  if (ws_bytes < kHeadBytes) return ELSAA_ERR_WORKSPACE;
  const void* const out[5] = {k, v, q_out, k_pages, v_pages};
  if (shared_start(out, 5, 3) || k_pages == q || v_pages == q) return ELSAA_ERR_INVALID_ARG;
  const int e = esize(p->dtype);
  auto take = [&](int i, int h, Strides* to) {
    return take_row_strides(strides ? strides + 2 * i : nullptr, p->rows, h, p->d, e, to);
  };
  if (!take(0, p->H, &a.sq) || !take(1, p->H, &a.sqo) || !take(2, p->Hkv, &a.sk) ||
      !take(3, p->Hkv, &a.sv) || !page_strides_of(p, page_strides, &a.skp, &a.svp))
    return ELSAA_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = q_out;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.page_table = page_table;
  a.starts = starts;
  a.lengths = lengths;
  a.seqs = p->seqs;
  a.page_size = p->page_size;
  a.pages = p->pages;
  a.table_width = p->table_width;
  return cuda_status(launch_paged_write(a, p->d, p->dtype == ELSAA_BF16, r->interleaved != 0,
                                        (cudaStream_t)stream));
}

elsaa_status elsaa_paged_attend(const elsaa_paged_params* p, const void* q,
                                const int64_t* strides, const void* k_pages, const void* v_pages,
                                const int64_t* page_strides, const int32_t* page_table,
                                const int32_t* starts, const int32_t* lengths, void* y, void* ws,
                                size_t ws_bytes, void* stream) {
  const elsaa_status st = check(p);
  if (st != ELSAA_OK) return st;
  if (!q || !k_pages || !v_pages || !page_table || !starts || !lengths || !y || !ws)
    return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {q, k_pages, v_pages, (const void*)y})
    if (!aligned16(x)) return ELSAA_ERR_INVALID_ARG;
  for (const void* x : {page_table, starts, lengths})
    if (!aligned4(x)) return ELSAA_ERR_INVALID_ARG;
  if (((uintptr_t)ws & 255) != 0) return ELSAA_ERR_INVALID_ARG;
  if (ws_bytes < elsaa_paged_workspace_bytes(p)) return ELSAA_ERR_WORKSPACE;
  if (y == q || y == k_pages || y == v_pages) return ELSAA_ERR_INVALID_ARG;
  AttendArgs a = {};
  const int e = esize(p->dtype);
  if (!take_row_strides(strides, p->rows, p->H, p->d, e, &a.sq) ||
      !take_row_strides(strides ? strides + 2 : nullptr, p->rows, p->H, p->d, e, &a.sy) ||
      !page_strides_of(p, page_strides, &a.sk, &a.sv))
    return ELSAA_ERR_INVALID_ARG;
  a.q = q;
  a.k = k_pages;
  a.v = v_pages;
  a.y = y;
  a.lengths = lengths;
  a.starts = starts;
  a.page_table = page_table;
  a.B = 1;
  a.H = p->H;
  a.Hkv = p->Hkv;
  a.N = p->rows;
  a.d = p->d;
  a.g = p->H / p->Hkv;
  a.window = p->window > 0 ? p->window : INT32_MAX;
  a.sinks = p->sinks;
  a.scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->d);
  a.err = (uint32_t*)ws;
  a.counters = (uint32_t*)((char*)ws + kCounters);
  a.scratch = (char*)ws + kHeadBytes;
  a.seqs = p->seqs;
  a.rows = p->rows;
  a.page_size = p->page_size;
  a.pages = p->pages;
  a.table_width = p->table_width;
  const bool bf16 = p->dtype == ELSAA_BF16;
  if (paged_decode_supported(p->d, bf16, p->rows, p->seqs, a.g))
    return cuda_status(launch_paged_decode(a, (cudaStream_t)stream));
  return cuda_status(attend_tc_supported(p->d, bf16)
                         ? launch_paged_tc(a, (cudaStream_t)stream)
                         : launch_paged_simt(a, bf16, (cudaStream_t)stream));
}

}  // extern "C"
