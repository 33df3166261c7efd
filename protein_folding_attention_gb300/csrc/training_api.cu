// C ABI of the training operators around the blocks (evoattn_block_norm,
// evoattn_block_norm_bwd, evoattn_grad_norm, evoattn_adamw): host-side
// validation and dispatch.  Every check happens before anything is enqueued;
// see include/evoattn.h for the contract.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "block_norm.h"
#include "evoattn.h"
#include "optim.h"

namespace evo {
namespace {

// One [B, I, J, C] operand as the caller gave it.
struct Rows4 {
  const void* p;
  const int64_t* s;
  evoattn_dtype dtype;
  bool output;
};

bool all_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p) return false;
  return true;
}

evoattn_status check_sizes(int B, int I, int J, int C, evoattn_dtype sd, evoattn_dtype d,
                           evoattn_norm_kind kind, float eps) {
  if (B < 1 || I < 1 || J < 1 || C < 1) return EVOATTN_ERR_INVALID_ARG;
  if (kind != EVOATTN_NORM_LAYER && kind != EVOATTN_NORM_RMS) return EVOATTN_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !(eps < INFINITY)) return EVOATTN_ERR_INVALID_ARG;
  const bool pair = (sd == EVOATTN_BF16 && d == EVOATTN_BF16) ||
                    (sd == EVOATTN_F32 && (d == EVOATTN_BF16 || d == EVOATTN_F32));
  if (!pair || C > kNormMaxC) return EVOATTN_ERR_UNSUPPORTED;
  const uint64_t limit = 0x7FFFFFFFull - (1u << 21);
  const uint64_t bi = (uint64_t)B * (uint64_t)I;  // < 2^62
  if (bi > limit || bi * (uint64_t)J > limit) return EVOATTN_ERR_UNSUPPORTED;
  return EVOATTN_OK;
}

// Strides and alignment of the operands that are given; rows of an output may
// not overlap, but for the axes along which `shared` (the gate) repeats one.
evoattn_status check_rows(std::initializer_list<Rows4> ops, const int (&n)[3], int C,
                          const int64_t* shared) {
  for (const Rows4& o : ops)
    if (o.p && !o.s) return EVOATTN_ERR_INVALID_ARG;
  for (const Rows4& o : ops) {
    if (!o.p) continue;
    for (int k = 0; k < 3; ++k) {
      if (n[k] == 1) continue;
      // (a span that fits 62 bits: no address computation overflows)
      if (o.s[k] < 0 || o.s[k] > (int64_t)1 << 58 || (__int128)o.s[k] * n[k] > (__int128)1 << 58)
        return EVOATTN_ERR_INVALID_ARG;
    }
    if (!o.output) continue;
    int axis[3], m = 0;
    for (int k = 0; k < 3; ++k)
      if (n[k] > 1 && !(shared && shared[k] == 0)) axis[m++] = k;
    std::sort(axis, axis + m, [&](int a, int b) { return o.s[a] < o.s[b]; });
    int64_t span = C;  // elements that the faster axes reach over
    for (int k = 0; k < m; ++k) {
      if (o.s[axis[k]] < span) return EVOATTN_ERR_INVALID_ARG;
      span += o.s[axis[k]] * (int64_t)(n[axis[k]] - 1);
    }
  }
  for (const Rows4& o : ops) {
    if (!o.p) continue;
    if (C > 1 && o.s[3] != 1) return EVOATTN_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(o.p) % (o.dtype == EVOATTN_BF16 ? 2 : 4)) return EVOATTN_ERR_ALIGNMENT;
  }
  return EVOATTN_OK;
}

bool floats_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 4) return false;
  return true;
}

RowOperand operand(const void* p, const int64_t* s) {
  RowOperand r{const_cast<void*>(p), {0, 0, 0}};
  if (p)
    for (int k = 0; k < 3; ++k) r.s[k] = s[k];
  return r;
}

// Reads the arguments of a packed call one after another.
class Words {
 public:
  struct Rows {
    void* p;
    const int64_t* s;
  };
  Words(const int64_t* w, int count) : w_(w), end_(w + count) {}
  Rows rows() {
    const int64_t* at = w_;
    w_ += 5;
    return Rows{reinterpret_cast<void*>(at[0]), at[0] ? at + 1 : nullptr};
  }
  template <typename T>
  T* pointer() { return reinterpret_cast<T*>(*w_++); }
  int integer() {
    const int64_t v = *w_++;
    if (v != (int64_t)(int)v) fits_ = false;
    return (int)v;
  }
  float real() {
    double d;
    memcpy(&d, w_++, sizeof(d));
    return (float)d;
  }
  size_t size() { return (size_t)*w_++; }
  bool complete() const { return fits_ && w_ == end_; }

 private:
  const int64_t *w_, *end_;
  bool fits_ = true;
};

evoattn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? EVOATTN_OK : EVOATTN_ERR_CUDA; }

}  // namespace
}  // namespace evo

using namespace evo;

extern "C" {

evoattn_status evoattn_block_norm(const void* x, const int64_t x_strides[4], const void* u,
                                  const int64_t u_strides[4], const void* gate,
                                  const int64_t gate_strides[4], const float* scale,
                                  const float* gamma_post, const float* beta_post,
                                  const float* gamma_pre, const float* beta_pre, void* x1,
                                  const int64_t x1_strides[4], void* y, const int64_t y_strides[4],
                                  int B, int I, int J, int C, evoattn_dtype stream_dtype,
                                  evoattn_dtype dtype, evoattn_norm_kind kind, float eps,
                                  cudaStream_t stream) {
  if (!x || (!u && !y) || (u != nullptr) != (x1 != nullptr)) return EVOATTN_ERR_INVALID_ARG;
  if (!u && !all_null({gate, scale, gamma_post, beta_post})) return EVOATTN_ERR_INVALID_ARG;
  if (!y && !all_null({gamma_pre, beta_pre})) return EVOATTN_ERR_INVALID_ARG;
  evoattn_status st = check_sizes(B, I, J, C, stream_dtype, dtype, kind, eps);
  if (st != EVOATTN_OK) return st;
  const int n[3] = {B, I, J};
  st = check_rows({{x, x_strides, stream_dtype, false}, {u, u_strides, dtype, false},
                   {gate, gate_strides, dtype, false}, {x1, x1_strides, stream_dtype, true},
                   {y, y_strides, dtype, true}}, n, C, nullptr);
  if (st != EVOATTN_OK) return st;
  if (!floats_aligned({scale, gamma_post, beta_post, gamma_pre, beta_pre})) return EVOATTN_ERR_ALIGNMENT;
  BlockNormCall c{};
  c.n[0] = B; c.n[1] = I; c.n[2] = J; c.C = C;
  c.rms = kind == EVOATTN_NORM_RMS;
  c.eps = eps;
  c.x = operand(x, x_strides);
  c.u = operand(u, u_strides);
  c.gate = operand(gate, gate_strides);
  c.x1 = operand(x1, x1_strides);
  c.y = operand(y, y_strides);
  c.scale = scale; c.gamma_post = gamma_post; c.beta_post = beta_post;
  c.gamma_pre = gamma_pre; c.beta_pre = beta_pre;
  if (stream_dtype == EVOATTN_BF16) return cuda_status(block_norm_fwd_bf16(c, stream));
  return cuda_status(dtype == EVOATTN_BF16 ? block_norm_fwd_mixed(c, stream) : block_norm_fwd_f32(c, stream));
}

size_t evoattn_block_norm_bwd_workspace_size(int C) {
  return C < 1 || C > kNormMaxC ? 0 : block_norm_bwd_workspace_bytes(C);
}

evoattn_status evoattn_block_norm_bwd(
    const void* dx1, const int64_t dx1_strides[4], const void* dy, const int64_t dy_strides[4],
    const void* x1, const int64_t x1_strides[4], const void* u, const int64_t u_strides[4],
    const void* gate, const int64_t gate_strides[4], const float* scale, const float* gamma_post,
    const float* beta_post, const float* gamma_pre, void* dx, const int64_t dx_strides[4],
    void* du, const int64_t du_strides[4], void* dgate, const int64_t dgate_strides[4],
    float* dscale, float* dgamma_post, float* dbeta_post, float* dgamma_pre, float* dbeta_pre,
    int B, int I, int J, int C, evoattn_dtype stream_dtype, evoattn_dtype dtype,
    evoattn_norm_kind kind, float eps, void* workspace, size_t workspace_bytes,
    cudaStream_t stream) {
  if ((!dx1 && !dy) || (!u && !dy)) return EVOATTN_ERR_INVALID_ARG;
  if ((dy != nullptr) != (x1 != nullptr) || (dy != nullptr) != (dx != nullptr)) return EVOATTN_ERR_INVALID_ARG;
  if ((u != nullptr) != (du != nullptr) || (gate != nullptr) != (dgate != nullptr))
    return EVOATTN_ERR_INVALID_ARG;
  if (!u && !all_null({gate, scale, gamma_post, beta_post, dscale, dgamma_post, dbeta_post}))
    return EVOATTN_ERR_INVALID_ARG;
  if (!dy && !all_null({gamma_pre, dgamma_pre, dbeta_pre})) return EVOATTN_ERR_INVALID_ARG;
  evoattn_status st = check_sizes(B, I, J, C, stream_dtype, dtype, kind, eps);
  if (st != EVOATTN_OK) return st;
  const int n[3] = {B, I, J};
  st = check_rows({{dx1, dx1_strides, stream_dtype, false}, {dy, dy_strides, dtype, false},
                   {x1, x1_strides, stream_dtype, false}, {u, u_strides, dtype, false},
                   {gate, gate_strides, dtype, false}, {dx, dx_strides, stream_dtype, true},
                   {du, du_strides, dtype, true}}, n, C, nullptr);
  if (st != EVOATTN_OK) return st;
  if (gate) {  // the gate's gradient repeats exactly the rows that the gate repeats
    st = check_rows({{dgate, dgate_strides, dtype, true}}, n, C, gate_strides);
    if (st != EVOATTN_OK) return st;
    for (int k = 0; k < 3; ++k)
      if (n[k] > 1 && (gate_strides[k] == 0) != (dgate_strides[k] == 0)) return EVOATTN_ERR_INVALID_ARG;
  }
  if (!floats_aligned({scale, gamma_post, beta_post, gamma_pre, dscale, dgamma_post, dbeta_post,
                       dgamma_pre, dbeta_pre}))
    return EVOATTN_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < block_norm_bwd_workspace_bytes(C) ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return EVOATTN_ERR_WORKSPACE;
  BlockNormCall c{};
  c.n[0] = B; c.n[1] = I; c.n[2] = J; c.C = C;
  c.rms = kind == EVOATTN_NORM_RMS;
  c.eps = eps;
  c.x = operand(x1, x1_strides);
  c.u = operand(u, u_strides);
  c.gate = operand(gate, gate_strides);
  c.dx1 = operand(dx1, dx1_strides);
  c.dy = operand(dy, dy_strides);
  c.dx = operand(dx, dx_strides);
  c.du = operand(du, du_strides);
  c.dgate = operand(dgate, dgate_strides);
  c.scale = scale; c.gamma_post = gamma_post; c.beta_post = beta_post; c.gamma_pre = gamma_pre;
  c.dscale = dscale; c.dgamma_post = dgamma_post; c.dbeta_post = dbeta_post;
  c.dgamma_pre = dgamma_pre; c.dbeta_pre = dbeta_pre;
  c.ws = static_cast<float*>(workspace);
  if (stream_dtype == EVOATTN_BF16) return cuda_status(block_norm_bwd_bf16(c, stream));
  return cuda_status(dtype == EVOATTN_BF16 ? block_norm_bwd_mixed(c, stream) : block_norm_bwd_f32(c, stream));
}

evoattn_status evoattn_block_norm_packed(const int64_t* words, cudaStream_t stream) {
  if (!words) return EVOATTN_ERR_INVALID_ARG;
  Words w(words, EVOATTN_BLOCK_NORM_WORDS);
  const Words::Rows x = w.rows(), u = w.rows(), gate = w.rows();
  float* prm[5];
  for (float*& p : prm) p = w.pointer<float>();
  const Words::Rows x1 = w.rows(), y = w.rows();
  int n[7];
  for (int& v : n) v = w.integer();
  const float eps = w.real();
  if (!w.complete()) return EVOATTN_ERR_INVALID_ARG;
  return evoattn_block_norm(x.p, x.s, u.p, u.s, gate.p, gate.s, prm[0], prm[1], prm[2], prm[3], prm[4],
                            x1.p, x1.s, y.p, y.s, n[0], n[1], n[2], n[3], (evoattn_dtype)n[4],
                            (evoattn_dtype)n[5], (evoattn_norm_kind)n[6], eps, stream);
}

evoattn_status evoattn_block_norm_bwd_packed(const int64_t* words, cudaStream_t stream) {
  if (!words) return EVOATTN_ERR_INVALID_ARG;
  Words w(words, EVOATTN_BLOCK_NORM_BWD_WORDS);
  const Words::Rows dx1 = w.rows(), dy = w.rows(), x1 = w.rows(), u = w.rows(), gate = w.rows();
  float* prm[4];
  for (float*& p : prm) p = w.pointer<float>();
  const Words::Rows dx = w.rows(), du = w.rows(), dgate = w.rows();
  float* grad[5];
  for (float*& p : grad) p = w.pointer<float>();
  int n[7];
  for (int& v : n) v = w.integer();
  const float eps = w.real();
  void* ws = w.pointer<void>();
  const size_t bytes = w.size();
  if (!w.complete()) return EVOATTN_ERR_INVALID_ARG;
  return evoattn_block_norm_bwd(dx1.p, dx1.s, dy.p, dy.s, x1.p, x1.s, u.p, u.s, gate.p, gate.s, prm[0],
                                prm[1], prm[2], prm[3], dx.p, dx.s, du.p, du.s, dgate.p, dgate.s, grad[0],
                                grad[1], grad[2], grad[3], grad[4], n[0], n[1], n[2], n[3],
                                (evoattn_dtype)n[4], (evoattn_dtype)n[5], (evoattn_norm_kind)n[6], eps,
                                ws, bytes, stream);
}

size_t evoattn_grad_norm_workspace_size(int count) {
  return count < 1 ? 0 : grad_norm_workspace_bytes(count);
}

static evoattn_status check_grads(const evoattn_adamw_tensor* t, int count,
                                  const evoattn_optim_state* state) {
  if (!t || count < 1 || !state) return EVOATTN_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0 || (t[i].n > 0 && !t[i].grad)) return EVOATTN_ERR_INVALID_ARG;
    if (t[i].grad_dtype != EVOATTN_BF16 && t[i].grad_dtype != EVOATTN_F32) return EVOATTN_ERR_UNSUPPORTED;
    if (t[i].n > (int64_t)1 << 40) return EVOATTN_ERR_UNSUPPORTED;
    if (t[i].n > 0 && reinterpret_cast<uintptr_t>(t[i].grad) % (t[i].grad_dtype == EVOATTN_BF16 ? 2 : 4))
      return EVOATTN_ERR_ALIGNMENT;
  }
  if (reinterpret_cast<uintptr_t>(state) % 8) return EVOATTN_ERR_ALIGNMENT;
  return EVOATTN_OK;
}

evoattn_status evoattn_grad_norm(const evoattn_adamw_tensor* tensors, int count, float max_norm,
                                 evoattn_optim_state* state, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  const evoattn_status st = check_grads(tensors, count, state);
  if (st != EVOATTN_OK) return st;
  if (!(max_norm > 0.f)) return EVOATTN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < grad_norm_workspace_bytes(count) ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return EVOATTN_ERR_WORKSPACE;
  return cuda_status(grad_norm(tensors, count, max_norm, state, workspace, stream));
}

evoattn_status evoattn_adamw(const evoattn_adamw_tensor* tensors, int count, float lr,
                             const float* lr_device, double beta1, double beta2, float eps,
                             int state_bits, unsigned flags, evoattn_optim_state* state,
                             cudaStream_t stream) {
  const evoattn_status st = check_grads(tensors, count, state);
  if (st != EVOATTN_OK) return st;
  if (!(lr >= 0.f) || !(lr < INFINITY) || !(beta1 >= 0.0 && beta1 < 1.0) ||
      !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= FLT_MIN) || !(eps < INFINITY))
    return EVOATTN_ERR_INVALID_ARG;
  if (flags & ~EVOATTN_ADAMW_CLIP) return EVOATTN_ERR_INVALID_ARG;
  if (state_bits != 32 && state_bits != 8) return EVOATTN_ERR_UNSUPPORTED;
  const bool narrow = state_bits == 8;
  for (int i = 0; i < count; ++i) {
    const evoattn_adamw_tensor& t = tensors[i];
    if (!(t.weight_decay >= 0.f) || !(t.weight_decay < INFINITY)) return EVOATTN_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.exp_avg || !t.exp_avg_sq) return EVOATTN_ERR_INVALID_ARG;
    if (narrow != (t.exp_avg_scale != nullptr) || narrow != (t.exp_avg_sq_scale != nullptr))
      return EVOATTN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < count; ++i) {
    const evoattn_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (!floats_aligned({t.param, t.exp_avg_scale, t.exp_avg_sq_scale}) ||
        (!narrow && !floats_aligned({t.exp_avg, t.exp_avg_sq})) ||
        reinterpret_cast<uintptr_t>(t.copy) % 2)
      return EVOATTN_ERR_ALIGNMENT;
  }
  if (reinterpret_cast<uintptr_t>(lr_device) % 4) return EVOATTN_ERR_ALIGNMENT;
  const AdamwScalars s{lr, lr_device, beta1, beta2, eps, (flags & EVOATTN_ADAMW_CLIP) != 0};
  return cuda_status(narrow ? adamw8(tensors, count, s, state, stream)
                            : adamw32(tensors, count, s, state, stream));
}

}  // extern "C"
