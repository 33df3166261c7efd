// C ABI of the 8-bit projection path (evoattn_dropout_add, evoattn_norm8,
// evoattn_norm8_bwd, evoattn_quantize8, evoattn_matmul8): host-side validation
// and dispatch.  Every check happens before anything is enqueued; see
// include/evoattn.h for the contract.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "evoattn.h"
#include "matmul8.h"
#include "norm8.h"
#include "quantize8.h"
#include "row_checks.h"
#include "scale8.cuh"
#include "sm103.h"

namespace evo {
namespace {

constexpr int64_t kMaxSpan = (int64_t)1 << 58;  // elements: no address computation overflows

bool to_int(int64_t v, int* out) {
  *out = (int)v;
  return v == (int64_t)*out;
}

evoattn_status shape_of(const int64_t (&n)[4], int (&rows)[3], int* C) {
  for (int64_t v : n)
    if (v < 1) return EVOATTN_ERR_INVALID_ARG;
  for (int k = 0; k < 3; ++k)
    if (!to_int(n[k], &rows[k])) return EVOATTN_ERR_UNSUPPORTED;
  return to_int(n[3], C) ? EVOATTN_OK : EVOATTN_ERR_UNSUPPORTED;
}

bool type_ok(int64_t d) { return d == EVOATTN_BF16 || d == EVOATTN_F32; }

Rows4 rows4(const evoattn_rows& r, int bytes, bool output) { return Rows4{r.p, r.s, bytes, output}; }

RowOperand operand(const evoattn_rows& r) { return evo::operand(r.p, r.s); }

// The dropout of a call; `given`: whether there is something to drop.
evoattn_status mask_of(const evoattn_dropout& d, bool given, const int (&n)[3], bool* drop, DropMask* m) {
  if (!(d.p >= 0.0) || !(d.p < 1.0) || d.site < 0 || d.site > (int64_t)UINT32_MAX || d.shared < 0 || d.shared > 7)
    return EVOATTN_ERR_INVALID_ARG;
  if (!given && d.p != 0.0) return EVOATTN_ERR_INVALID_ARG;
  *drop = d.p > 0.0;
  if (!*drop) return EVOATTN_OK;
  if (!d.rng) return EVOATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(d.rng) % 8) return EVOATTN_ERR_ALIGNMENT;
  m->rng = d.rng;
  m->site = (uint32_t)d.site;
  m->threshold = (uint32_t)std::min(floor(d.p * 4294967296.0 + 0.5), 4294967295.0);
  m->scale = (float)(1.0 / (1.0 - d.p));
  int64_t step = 1;
  for (int k = 2; k >= 0; --k) {
    m->s[k] = d.shared >> k & 1 ? 0 : step;
    if (!(d.shared >> k & 1)) step *= n[k];
  }
  return EVOATTN_OK;
}

// Merges neighbouring row axes where every stride array in `ops` (each once;
// NULL for an operand that is not given) allows it, so that a kernel divides a
// row's index no more often than it has to.
void merge_axes(int (&n)[3], std::initializer_list<int64_t*> ops) {
  const auto merge = [&](int a, int b) {
    if (n[a] > 1 && n[b] > 1)
      for (const int64_t* s : ops)
        if (s && s[a] != (int64_t)n[b] * s[b]) return;
    for (int64_t* s : ops) {
      if (!s) continue;
      if (n[b] == 1) s[b] = n[a] == 1 ? 0 : s[a];
      s[a] = 0;
    }
    n[b] *= n[a];
    n[a] = 1;
  };
  merge(0, 1);
  merge(1, 2);
  merge(0, 1);
}

// Exchanges the axes I and J where J is the outer one in memory for all of `by`, so
// that rows are walked as they lie (rows of the ending node's views would each
// come from another DRAM page).  `ops`: every stride array, `by` among them; NULL
// for an operand that is not given.  Returns whether it did.
bool rows_as_they_lie(int (&n)[3], std::initializer_list<const int64_t*> by, std::initializer_list<int64_t*> ops) {
  if (n[1] == 1 || n[2] == 1) return false;
  for (const int64_t* s : by)
    if (s && s[1] >= s[2]) return false;
  for (int64_t* s : ops)
    if (s) std::swap(s[1], s[2]);
  std::swap(n[1], n[2]);
  return true;
}

// Scales of an output: distinct places for all of them.
evoattn_status check_scales(const evoattn_rows& r, const int (&n)[3], int groups) {
  const int64_t extent[4] = {n[0], n[1], n[2], groups};
  int axis[4], m = 0;
  for (int k = 0; k < 4; ++k) {
    if (extent[k] == 1) continue;
    if (r.s[k] < 0 || r.s[k] > kMaxSpan || (__int128)r.s[k] * extent[k] > kMaxSpan) return EVOATTN_ERR_INVALID_ARG;
    axis[m++] = k;
  }
  std::sort(axis, axis + m, [&](int a, int b) { return r.s[a] < r.s[b]; });
  int64_t span = 1;
  for (int k = 0; k < m; ++k) {
    if (r.s[axis[k]] < span) return EVOATTN_ERR_INVALID_ARG;
    span += r.s[axis[k]] * (extent[axis[k]] - 1);
  }
  return EVOATTN_OK;
}

// A matrix of bytes with 16-byte aligned rows.
evoattn_status check_codes(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  if (ld < cols || ld > (int64_t)1 << 39 || (__int128)ld * rows > kMaxSpan) return EVOATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % 16 || ld % 16) return EVOATTN_ERR_ALIGNMENT;
  return EVOATTN_OK;
}

bool scale_strides_ok(int64_t row, int64_t group, int64_t rows, int64_t groups) {
  return row >= 0 && group >= 0 && row <= kMaxSpan && group <= kMaxSpan && (__int128)row * rows <= kMaxSpan &&
         (__int128)group * groups <= kMaxSpan;
}
// ... of an output: distinct places.
bool scales_distinct(int64_t row, int64_t group, int64_t rows, int64_t groups) {
  if (!scale_strides_ok(row, group, rows, groups)) return false;
  if (rows > 1 && row < 1) return false;
  if (groups > 1 && group < 1) return false;
  return rows == 1 || groups == 1 || row >= group * groups || group >= row * rows;
}

int64_t groups_of(int64_t k) { return (k + kGroup8 - 1) / kGroup8; }

evoattn_status operand_of(const evoattn_operand8& o, int rows, int K, Operand8* to) {
  if (!o.codes || !o.scales || (o.rows_per_scale != 1 && o.rows_per_scale != kGroup8)) return EVOATTN_ERR_INVALID_ARG;
  if (!scale_strides_ok(o.s_row, o.s_group, rows, groups_of(K))) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_status st = check_codes(o.codes, o.ld, rows, K);
  if (st != EVOATTN_OK) return st;
  *to = Operand8{o.codes, o.ld, o.scales, o.s_row, o.s_group, o.rows_per_scale == 1 ? 0 : 7};
  return EVOATTN_OK;
}

bool sm_count(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && *sms > 0;
}

}  // namespace
}  // namespace evo

using namespace evo;

extern "C" {

evoattn_status evoattn_dropout_add(const evoattn_dropout_add_args* args, cudaStream_t stream) {
  if (!args || !args->u.p || !args->out.p) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_dropout_add_args& a = *args;
  int n[3], C;
  evoattn_status st = shape_of(a.n, n, &C);
  if (st != EVOATTN_OK) return st;
  if (!type_ok(a.stream_dtype) || !type_ok(a.dtype)) return EVOATTN_ERR_UNSUPPORTED;
  // (any pair of types: the sizes are checked as for two of the same)
  st = check_sizes(n[0], n[1], n[2], C, EVOATTN_F32, EVOATTN_F32, EVOATTN_NORM_LAYER, 1.f);
  if (st != EVOATTN_OK) return st;
  if ((uint64_t)n[0] * n[1] * n[2] * (uint64_t)((C + 7) / 8) > 0xFFFFFFFFull) return EVOATTN_ERR_UNSUPPORTED;
  const int wide = bytes_of((evoattn_dtype)a.stream_dtype), narrow = bytes_of((evoattn_dtype)a.dtype);
  st = check_rows({rows4(a.x, wide, false), rows4(a.u, narrow, false), rows4(a.out, wide, true)}, n, C, nullptr);
  if (st != EVOATTN_OK) return st;
  Norm8Call c{};
  st = mask_of(a.drop, true, n, &c.drop, &c.mask);
  if (st != EVOATTN_OK) return st;
  c.x = operand(a.x);
  c.u = operand(a.u);
  c.x1 = operand(a.out);
  c.C = C;
  int64_t *const x = c.x.p ? c.x.s : nullptr, *const mask = c.drop ? c.mask.s : nullptr;
  c.turned = rows_as_they_lie(n, {x, c.u.s, c.x1.s}, {x, c.u.s, c.x1.s, mask});
  std::copy(n, n + 3, c.given);
  merge_axes(n, {x, c.u.s, c.x1.s});
  std::copy(n, n + 3, c.n);
  if (a.stream_dtype == EVOATTN_BF16)
    return cuda_status(a.dtype == EVOATTN_BF16 ? dropout_add_bf16(c, stream) : dropout_add_narrow(c, stream));
  return cuda_status(a.dtype == EVOATTN_BF16 ? dropout_add_mixed(c, stream) : dropout_add_f32(c, stream));
}

evoattn_status evoattn_norm8(const evoattn_norm8_args* args, cudaStream_t stream) {
  if (!args || !args->x.p || !args->codes.p || !args->scales.p) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_norm8_args& a = *args;
  if ((a.u.p != nullptr) != (a.x1.p != nullptr)) return EVOATTN_ERR_INVALID_ARG;
  int n[3], C;
  evoattn_status st = shape_of(a.n, n, &C);
  if (st != EVOATTN_OK) return st;
  if (!type_ok(a.stream_dtype) || !type_ok(a.dtype)) return EVOATTN_ERR_UNSUPPORTED;
  if (a.kind != EVOATTN_NORM_LAYER && a.kind != EVOATTN_NORM_RMS) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_dtype sd = (evoattn_dtype)a.stream_dtype, d = (evoattn_dtype)a.dtype;
  st = check_sizes(n[0], n[1], n[2], C, sd, d, (evoattn_norm_kind)a.kind, (float)a.eps);
  if (st != EVOATTN_OK) return st;
  st = check_rows({rows4(a.x, bytes_of(sd), false), rows4(a.u, bytes_of(d), false),
                   rows4(a.x1, bytes_of(sd), true), rows4(a.codes, 1, true)}, n, C, nullptr);
  if (st == EVOATTN_OK) st = check_scales(a.scales, n, (int)groups_of(C));
  if (st != EVOATTN_OK) return st;
  if (!floats_aligned({a.gamma, a.beta})) return EVOATTN_ERR_ALIGNMENT;
  Norm8Call c{};
  st = mask_of(a.drop, a.u.p != nullptr, n, &c.drop, &c.mask);
  if (st != EVOATTN_OK) return st;
  c.x = operand(a.x);
  c.u = operand(a.u);
  c.x1 = operand(a.x1);
  c.codes = static_cast<uint8_t*>(a.codes.p);
  c.scales = static_cast<uint8_t*>(a.scales.p);
  for (int k = 0; k < 3; ++k) { c.codes_s[k] = a.codes.s[k]; c.scales_s[k] = a.scales.s[k]; }
  c.scales_g = groups_of(C) > 1 ? a.scales.s[3] : 0;
  c.gamma = a.gamma;
  c.beta = a.beta;
  c.C = C;
  c.rms = a.kind == EVOATTN_NORM_RMS;
  c.eps = (float)a.eps;
  int64_t *const u = c.u.p ? c.u.s : nullptr, *const x1 = c.u.p ? c.x1.s : nullptr;
  c.turned = rows_as_they_lie(n, {c.x.s, u, x1}, {c.x.s, u, x1, c.codes_s, c.scales_s, c.drop ? c.mask.s : nullptr});
  std::copy(n, n + 3, c.given);
  merge_axes(n, {c.x.s, u, x1, c.codes_s, c.scales_s});
  std::copy(n, n + 3, c.n);
  if (sd == EVOATTN_BF16) return cuda_status(norm8_fwd_bf16(c, stream));
  return cuda_status(d == EVOATTN_BF16 ? norm8_fwd_mixed(c, stream) : norm8_fwd_f32(c, stream));
}

size_t evoattn_norm8_bwd_workspace_size(int C) {
  return C < 1 || C > kNormMaxC ? 0 : norm8_bwd_workspace_bytes(C);
}

evoattn_status evoattn_norm8_bwd(const evoattn_norm8_bwd_args* args, cudaStream_t stream) {
  if (!args || !args->dy.p || !args->x1.p || !args->dx.p) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_norm8_bwd_args& a = *args;
  int n[3], C;
  evoattn_status st = shape_of(a.n, n, &C);
  if (st != EVOATTN_OK) return st;
  if (!type_ok(a.stream_dtype) || !type_ok(a.dtype)) return EVOATTN_ERR_UNSUPPORTED;
  if (a.kind != EVOATTN_NORM_LAYER && a.kind != EVOATTN_NORM_RMS) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_dtype sd = (evoattn_dtype)a.stream_dtype, d = (evoattn_dtype)a.dtype;
  st = check_sizes(n[0], n[1], n[2], C, sd, d, (evoattn_norm_kind)a.kind, (float)a.eps);
  if (st != EVOATTN_OK) return st;
  st = check_rows({rows4(a.dx1, bytes_of(sd), false), rows4(a.dy, bytes_of(d), false),
                   rows4(a.x1, bytes_of(sd), false), rows4(a.dx, bytes_of(sd), true),
                   rows4(a.du, bytes_of(d), true)}, n, C, nullptr);
  if (st != EVOATTN_OK) return st;
  if (!floats_aligned({a.gamma, a.dgamma, a.dbeta})) return EVOATTN_ERR_ALIGNMENT;
  Norm8Call c{};
  st = mask_of(a.drop, a.du.p != nullptr, n, &c.drop, &c.mask);
  if (st != EVOATTN_OK) return st;
  if (!a.workspace || a.workspace_bytes < 0 || (size_t)a.workspace_bytes < norm8_bwd_workspace_bytes(C) ||
      reinterpret_cast<uintptr_t>(a.workspace) % 256)
    return EVOATTN_ERR_WORKSPACE;
  c.dx1 = operand(a.dx1);
  c.dy = operand(a.dy);
  c.x1 = operand(a.x1);
  c.dx = operand(a.dx);
  c.du = operand(a.du);
  c.gamma = a.gamma;
  c.dgamma = a.dgamma;
  c.dbeta = a.dbeta;
  c.ws = static_cast<float*>(a.workspace);
  c.C = C;
  c.rms = a.kind == EVOATTN_NORM_RMS;
  c.eps = (float)a.eps;
  int64_t *const dx1 = c.dx1.p ? c.dx1.s : nullptr, *const du = c.du.p ? c.du.s : nullptr;
  c.turned = rows_as_they_lie(n, {c.x1.s, c.dy.s, c.dx.s, dx1, du},
                              {c.x1.s, c.dy.s, c.dx.s, dx1, du, c.drop ? c.mask.s : nullptr});
  std::copy(n, n + 3, c.given);
  merge_axes(n, {c.x1.s, c.dy.s, c.dx.s, dx1, du});
  std::copy(n, n + 3, c.n);
  if (sd == EVOATTN_BF16) return cuda_status(norm8_bwd_bf16(c, stream));
  return cuda_status(d == EVOATTN_BF16 ? norm8_bwd_mixed(c, stream) : norm8_bwd_f32(c, stream));
}

evoattn_status evoattn_quantize8(const evoattn_quantize8_args* args, cudaStream_t stream) {
  if (!args) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_quantize8_args& a = *args;
  if (!a.x || (!a.codes && !a.codes_t) || a.R < 1 || a.K < 1) return EVOATTN_ERR_INVALID_ARG;
  const int64_t rg = groups_of(a.R), kg = groups_of(a.K);
  const bool blocks = a.blocks != 0;
  if (blocks ? (!a.scales || a.scales_t) : ((a.codes != nullptr) != (a.scales != nullptr) ||
                                            (a.codes_t != nullptr) != (a.scales_t != nullptr)))
    return EVOATTN_ERR_INVALID_ARG;
  if (!type_ok(a.dtype)) return EVOATTN_ERR_UNSUPPORTED;
  if (a.R > (int64_t)1 << 40 || a.K > (int64_t)1 << 40 || (__int128)rg * kg > 0x3FFFFFFF) return EVOATTN_ERR_UNSUPPORTED;
  const int bytes = bytes_of((evoattn_dtype)a.dtype);
  if (a.R > 1 && (a.ld < 0 || a.ld > kMaxSpan || (__int128)a.ld * a.R > kMaxSpan)) return EVOATTN_ERR_INVALID_ARG;
  if (a.scales && !scales_distinct(a.s_row, a.s_group, blocks ? rg : a.R, kg)) return EVOATTN_ERR_INVALID_ARG;
  if (a.scales_t && !scales_distinct(a.st_row, a.st_group, a.K, rg)) return EVOATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a.x) % bytes) return EVOATTN_ERR_ALIGNMENT;
  evoattn_status st = a.codes ? check_codes(a.codes, a.ldc, a.R, a.K) : EVOATTN_OK;
  if (st == EVOATTN_OK && a.codes_t) st = check_codes(a.codes_t, a.ldt, a.K, a.R);
  if (st != EVOATTN_OK) return st;
  Quantize8Call c{};
  c.x = a.x; c.R = a.R; c.K = a.K;
  c.ld = a.R > 1 ? a.ld : 0;
  c.blocks = blocks;
  c.codes = static_cast<uint8_t*>(a.codes); c.ldc = a.ldc;
  c.scales = a.scales; c.s_row = a.s_row; c.s_group = a.s_group;
  c.codes_t = static_cast<uint8_t*>(a.codes_t); c.ldt = a.ldt;
  c.scales_t = a.scales_t; c.st_row = a.st_row; c.st_group = a.st_group;
  return cuda_status(quantize8(c, a.dtype == EVOATTN_F32, stream));
}

size_t evoattn_matmul8_workspace_size(int M, int N, int K) {
  int sms = 0;
  if (M < 1 || N < 1 || K < 1 || !sm_count(&sms)) return 0;
  return matmul8_workspace_bytes(M, N, K, sms);
}

evoattn_status evoattn_matmul8(const evoattn_matmul8_args* args, cudaStream_t stream) {
  if (!args) return EVOATTN_ERR_INVALID_ARG;
  const evoattn_matmul8_args& a = *args;
  if (a.M < 1 || a.N < 1 || a.K < 1 || !a.out) return EVOATTN_ERR_INVALID_ARG;
  Matmul8Call c{};
  const int64_t most = 0x7FFFFFFF - 256;
  if (a.M > most || a.N > most || a.K > most || !type_ok(a.dtype)) return EVOATTN_ERR_UNSUPPORTED;
  c.M = (int)a.M; c.N = (int)a.N; c.K = (int)a.K;
  c.f32 = a.dtype == EVOATTN_F32;
  if (a.M > 1 && (a.ld_out < a.N || a.ld_out > kMaxSpan || (__int128)a.ld_out * a.M > kMaxSpan))
    return EVOATTN_ERR_INVALID_ARG;
  if (a.add && a.M > 1 &&
      ((a.ld_add != 0 && a.ld_add < a.N) || a.ld_add > kMaxSpan || (__int128)a.ld_add * a.M > kMaxSpan))
    return EVOATTN_ERR_INVALID_ARG;
  evoattn_status st = operand_of(a.a, c.M, c.K, &c.a);
  if (st == EVOATTN_OK) st = operand_of(a.b, c.N, c.K, &c.b);
  if (st != EVOATTN_OK) return st;
  const int bytes = c.f32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(a.out) % bytes || reinterpret_cast<uintptr_t>(a.add) % bytes)
    return EVOATTN_ERR_ALIGNMENT;
  int sms = 0;
  if (!sm_count(&sms) || !wait_config(&c.wait)) return EVOATTN_ERR_CUDA;
  const Matmul8Plan plan = matmul8_plan(c.M, c.N, c.K, sms);
  if ((__int128)plan.tiles_p * plan.tiles_q * plan.splits > most) return EVOATTN_ERR_UNSUPPORTED;
  const size_t need = matmul8_workspace_bytes(c.M, c.N, c.K, sms);
  if (need && (!a.workspace || a.workspace_bytes < 0 || (size_t)a.workspace_bytes < need ||
               reinterpret_cast<uintptr_t>(a.workspace) % 256))
    return EVOATTN_ERR_WORKSPACE;
  c.out = a.out;
  c.ld_out = a.M > 1 ? a.ld_out : 0;
  c.add = a.add;
  c.ld_add = a.add && a.M > 1 ? a.ld_add : 0;
  c.ws = static_cast<float*>(a.workspace);
  bool tmap_ok = true;
  const cudaError_t e = matmul8(c, plan, sms, stream, &tmap_ok);
  if (!tmap_ok) return EVOATTN_ERR_ALIGNMENT;
  return cuda_status(e);
}

}  // extern "C"
