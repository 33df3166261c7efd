// Checks of row operands that the C ABI's entry points share.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "block_norm.h"
#include "evoattn.h"

namespace evo {

// One [B, I, J, C] operand as the caller gave it.
struct Rows4 {
  const void* p;
  const int64_t* s;
  int bytes;  // of an element
  bool output;
};

inline bool all_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p) return false;
  return true;
}

inline evoattn_status check_sizes(int B, int I, int J, int C, evoattn_dtype sd, evoattn_dtype d,
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
inline evoattn_status check_rows(std::initializer_list<Rows4> ops, const int (&n)[3], int C,
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
    if (reinterpret_cast<uintptr_t>(o.p) % o.bytes) return EVOATTN_ERR_ALIGNMENT;
  }
  return EVOATTN_OK;
}

inline bool floats_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 4) return false;
  return true;
}

inline RowOperand operand(const void* p, const int64_t* s) {
  RowOperand r{const_cast<void*>(p), {0, 0, 0}};
  if (p)
    for (int k = 0; k < 3; ++k) r.s[k] = s[k];
  return r;
}

inline evoattn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? EVOATTN_OK : EVOATTN_ERR_CUDA; }

inline int bytes_of(evoattn_dtype d) { return d == EVOATTN_BF16 ? 2 : 4; }

}  // namespace evo
