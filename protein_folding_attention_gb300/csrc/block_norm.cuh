// The block norm on sm_103a: the norm after a block, its gate and residual
// scale, and the norm before the next block, in one pass over the rows, and
// the gradients of all of them in one pass.
//
// For every row r of C channels (u, gate, scale and the norm parameters are
// optional; s = sigmoid; n(v) is layer or root-mean-square normalisation):
//
//   x1 = x + scale * s(gate) * n(u; gamma_post, beta_post)
//   y  = n(x1; gamma_pre, beta_pre)            (of the unrounded x1)
//
// Backward, from x1 as the forward stored it (its statistics are recomputed:
// the row is in registers anyway, and saved statistics would have to be read):
//
//   h = (x1 - mean) rstd       a = dy gamma_pre
//   D = dx1 + rstd (a - mean(a) - h mean(a h))             -> dx
//   k = (u - mean) rstd        w = k gamma_post + beta_post,  q = s(gate)
//   dscale = sum D q w         dgate = D scale w q (1 - q)    e = D scale q
//   dgamma_post = sum e k      dbeta_post = sum e             b = e gamma_post
//   du = rstd (b - mean(b) - k mean(b k))
//   dgamma_pre = sum dy h      dbeta_pre = sum dy
//
// (rms: mean = 0 and no mean(a), mean(b) terms.)  Everything is held in fp32;
// each stored tensor is rounded once.  Bound by HBM: 10 bytes per element
// forward and 16 backward in bf16, against about 20 and 50 fp32 operations.
//
// Layout: a row belongs to a group of G threads, 8 channels each, so that a
// bf16 row is one 16-byte access per thread and its values stay in registers
// from load to store.  G = 8, 16 or 32 lanes of a warp up to C = 256 (sums by
// shuffles); above that W warps (sums by shuffles, then through shared memory
// with one named barrier per sum).  Persistent CTAs walk the rows, each thread
// keeping its channels' parameters, and in the backward the parameter
// gradients of its rows, in registers; the next row is loaded while the
// current one is worked on.  The CTAs' sums go to the workspace and a second
// kernel adds them in a fixed order: repeated calls give the same bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "block_norm.h"

namespace evo {
namespace norm {

constexpr int kE = 8;          // channels per thread
constexpr int kThreads = 256;  // threads of a CTA at most, where a row takes at most 8 warps

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
// n / d for n < 2^31 by a multiplication (d fixed per launch).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  const uint64_t m = ((1ull << 32) * ((1ull << l) - d)) / d + 1;
  return FastDiv{d, (uint32_t)m, l};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}

struct Rows {
  FastDiv d2, d1;  // extents of the innermost and the middle row axis
  bool flat;       // one row axis only
};
struct Operand {
  char* p;
  int64_t s0, s1, s2;  // bytes
};
struct RowPos {
  uint32_t i0, i1, i2;
};
__device__ __forceinline__ RowPos row_pos(const Rows& R, uint32_t row) {
  if (R.flat) return RowPos{0, 0, row};
  const uint32_t a = div_by(row, R.d2);
  const uint32_t b = div_by(a, R.d1);
  return RowPos{b, a - b * R.d1.d, row - a * R.d2.d};
}
__device__ __forceinline__ char* row_ptr(const Operand& o, const RowPos& r, bool flat) {
  char* p = o.p + r.i2 * o.s2;
  if (!flat) p += r.i1 * o.s1 + r.i0 * o.s0;
  return p;
}

struct Params {
  Rows rows_of;
  uint32_t rows;
  int C;
  int lanes;      // threads of a row's group (a multiple of 32 where it spans warps)
  bool rms;
  float eps, inv_c;
  Operand x, u, gate, x1, y, dx1, dy, dx, du, dgate;
  const float *scale, *gamma_post, *beta_post, *gamma_pre, *beta_pre;
  float* out[5];  // dscale, dgamma_post, dbeta_post, dgamma_pre, dbeta_pre
  float* part;    // [CTAs][5][C], or out[] itself when there is one CTA
  // a gate row shared by `share` consecutive rows: `segs` items of at most
  // `seg_rows` rows each per gate row
  uint32_t share, segs, seg_rows, items;
  bool by_cta;       // an item's rows are spread over the CTA (else one group walks them)
  float* gate_part;  // [items][C] where segs > 1
};

// ---------------------------------------------------------------------------
// a thread's 8 channels of a row
// ---------------------------------------------------------------------------
template <typename T, bool VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, true> {
  uint4 v;
};
template <>
struct Raw<float, true> {
  float4 a, b;
};
template <>
struct Raw<__nv_bfloat16, false> {
  __nv_bfloat16 v[kE];
};
template <>
struct Raw<float, false> {
  float v[kE];
};

// VEC: channels 8 * lane + e, with C a multiple of 8 and 16-byte aligned rows.
// Otherwise channels e * lanes + lane, one element per access.
template <bool VEC>
__device__ __forceinline__ int channel(int lane, int lanes, int e) {
  return VEC ? lane * kE + e : e * lanes + lane;
}

__device__ __forceinline__ void load(Raw<__nv_bfloat16, true>& r, const char* row, int lane, int, int) {
  r.v = *(reinterpret_cast<const uint4*>(row) + lane);
}
__device__ __forceinline__ void load(Raw<float, true>& r, const char* row, int lane, int, int) {
  const float4* p = reinterpret_cast<const float4*>(row) + 2 * lane;
  r.a = p[0];
  r.b = p[1];
}
template <typename T>
__device__ __forceinline__ void load(Raw<T, false>& r, const char* row, int lane, int lanes, int C) {
  const T* p = reinterpret_cast<const T*>(row);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int c = e * lanes + lane;
    r.v[e] = c < C ? p[c] : T(0.f);
  }
}

__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, true>& r, float (&v)[kE]) {
  v[0] = lo_bf16(r.v.x); v[1] = hi_bf16(r.v.x); v[2] = lo_bf16(r.v.y); v[3] = hi_bf16(r.v.y);
  v[4] = lo_bf16(r.v.z); v[5] = hi_bf16(r.v.z); v[6] = lo_bf16(r.v.w); v[7] = hi_bf16(r.v.w);
}
__device__ __forceinline__ void widen(const Raw<float, true>& r, float (&v)[kE]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw<T, false>& r, float (&v)[kE]) {
#pragma unroll
  for (int e = 0; e < kE; ++e) v[e] = static_cast<float>(r.v[e]);
}

template <typename T, bool VEC>
struct Store;
template <>
struct Store<__nv_bfloat16, true> {
  static __device__ __forceinline__ void put(char* row, int lane, int, int, const float (&v)[kE]) {
    *(reinterpret_cast<uint4*>(row) + lane) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
};
template <>
struct Store<float, true> {
  static __device__ __forceinline__ void put(char* row, int lane, int, int, const float (&v)[kE]) {
    float4* p = reinterpret_cast<float4*>(row) + 2 * lane;
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <typename T>
struct Store<T, false> {
  static __device__ __forceinline__ void put(char* row, int lane, int lanes, int C, const float (&v)[kE]) {
    T* p = reinterpret_cast<T*>(row);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = e * lanes + lane;
      if (c < C) p[c] = static_cast<T>(v[e]);
    }
  }
};

// A thread's channels of a parameter vector (`absent` without one).
template <bool VEC>
__device__ __forceinline__ void param(const float* p, float absent, int lane, int lanes, int C,
                                      float (&v)[kE]) {
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int c = channel<VEC>(lane, lanes, e);
    v[e] = c < C ? (p ? p[c] : absent) : 0.f;
  }
}

// ---------------------------------------------------------------------------
// sums over a row's group
// ---------------------------------------------------------------------------
// G lanes of a warp, or (G = 0) several warps: then every warp leaves its sum
// in shared memory and reads all of them behind one barrier.  Two buffers take
// turns, so that a sum's values are read before the barrier that precedes
// their buffer's next use.
constexpr int kMaxWarps = 16;
struct GroupSum {
  float2* buf;   // [2][kMaxWarps]
  int warps, warp, barrier, turn;
};

template <int G>
__device__ __forceinline__ float2 group_sum(float2 v, GroupSum& g) {
#pragma unroll
  for (int o = (G == 0 ? 32 : G) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (G == 0) {
    float2* b = g.buf + (g.turn ? kMaxWarps : 0);
    g.turn ^= 1;
    if ((threadIdx.x & 31) == 0) b[g.warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(g.barrier), "r"(g.warps * 32) : "memory");
    v = make_float2(0.f, 0.f);
    for (int i = 0; i < g.warps; ++i) {
      v.x += b[i].x;
      v.y += b[i].y;
    }
  }
  return v;
}

// What a thread knows of its group.
struct Group {
  int lane, lanes;   // place in the row's group
  int slot, slots;   // the group's place in the CTA
  bool act;          // VEC: the thread has channels
  GroupSum sum;
};

template <int G, bool VEC>
__device__ __forceinline__ Group make_group(const Params& p, float2 (*smem)[2 * kMaxWarps]) {
  Group g;
  if constexpr (G > 0) {
    g.lanes = G;
    g.slots = (int)blockDim.x / G;
    g.slot = (int)threadIdx.x / G;
    g.lane = (int)threadIdx.x % G;
    g.sum = GroupSum{nullptr, 1, 0, 0, 0};
  } else {
    g.lanes = p.lanes;
    g.slots = (int)blockDim.x / p.lanes;
    g.slot = (int)threadIdx.x / p.lanes;
    g.lane = (int)threadIdx.x - g.slot * p.lanes;
    g.sum = GroupSum{smem[g.slot], p.lanes / 32, g.lane / 32, 1 + g.slot, 0};
  }
  g.act = VEC ? g.lane * kE < p.C : true;
  return g;
}

// Whether this thread's channel e exists (VEC: all or none do, see Group::act).
template <bool VEC>
__device__ __forceinline__ bool has(const Group& g, int e, int C) {
  return VEC ? true : e * g.lanes + g.lane < C;
}

// Statistics of one or two rows at once (the second where `two`): mean (0 for
// rms) and 1 / sqrt(variance + eps); v becomes (v - mean) * rstd.  Two passes
// over registers, the deviations squared after the mean is removed.
template <int G, bool VEC, bool TWO>
__device__ __forceinline__ float2 standardise(float (&a)[kE], float (&b)[kE], Group& g,
                                              const Params& p) {
  float2 mean = make_float2(0.f, 0.f);
  if (!p.rms) {
    float2 s = make_float2(0.f, 0.f);
    if (g.act) {  // (without VEC, absent channels hold zeros)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        s.x += a[e];
        if (TWO) s.y += b[e];
      }
    }
    mean = group_sum<G>(s, g.sum);
    mean.x *= p.inv_c;
    mean.y *= p.inv_c;
  }
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const bool ok = has<VEC>(g, e, p.C);
    a[e] = ok ? a[e] - mean.x : 0.f;
    s.x = fmaf(a[e], a[e], s.x);
    if (TWO) {
      b[e] = ok ? b[e] - mean.y : 0.f;
      s.y = fmaf(b[e], b[e], s.y);
    }
  }
  if (!g.act) s = make_float2(0.f, 0.f);
  s = group_sum<G>(s, g.sum);
  const float2 r = make_float2(rsqrtf(fmaf(s.x, p.inv_c, p.eps)), rsqrtf(fmaf(s.y, p.inv_c, p.eps)));
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    a[e] *= r.x;
    if (TWO) b[e] *= r.y;
  }
  return r;
}

__device__ __forceinline__ float sigmoid(float v) {
  return __fdividef(1.f, 1.f + __expf(-v));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE>
__global__ void __launch_bounds__(G == 0 ? 512 : kThreads)
    k_block_norm_fwd(const __grid_constant__ Params p) {
  __shared__ float2 sums[8][2 * kMaxWarps];
  Group g = make_group<G, VEC>(p, sums);
  const int C = p.C;
  const bool flat = p.rows_of.flat, gated = POST && p.gate.p != nullptr;

  // scale folded into the post-norm's parameters
  float g1[kE], b1[kE], g2[kE], b2[kE];
  if (POST) {
    float s[kE];
    param<VEC>(p.scale, 1.f, g.lane, g.lanes, C, s);
    param<VEC>(p.gamma_post, 1.f, g.lane, g.lanes, C, g1);
    param<VEC>(p.beta_post, 0.f, g.lane, g.lanes, C, b1);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      g1[e] *= s[e];
      b1[e] *= s[e];
    }
  }
  if (PRE) {
    param<VEC>(p.gamma_pre, 1.f, g.lane, g.lanes, C, g2);
    param<VEC>(p.beta_pre, 0.f, g.lane, g.lanes, C, b2);
  }

  struct In {
    Raw<TS, VEC> x;
    Raw<TI, VEC> u, gate;
  };
  auto fetch = [&](In& in, uint32_t row) {
    const RowPos r = row_pos(p.rows_of, row);
    if (!g.act) return;
    load(in.x, row_ptr(p.x, r, flat), g.lane, g.lanes, C);
    if (POST) {
      load(in.u, row_ptr(p.u, r, flat), g.lane, g.lanes, C);
      if (gated) load(in.gate, row_ptr(p.gate, r, flat), g.lane, g.lanes, C);
    }
  };

  // every thread of a warp (or of a row's warps) takes part in the sums, so
  // all groups of a CTA make the same number of turns
  const uint32_t step = gridDim.x * g.slots;
  uint32_t first = blockIdx.x * g.slots;
  In cur{}, nxt{};
  if (first + g.slot < p.rows) fetch(cur, first + g.slot);
  for (; first < p.rows; first += step) {
    const uint32_t row = first + g.slot;
    const bool live = row < p.rows;
    if (row + step < p.rows) fetch(nxt, row + step);
    const RowPos r = row_pos(p.rows_of, live ? row : 0);
    float x[kE];
    widen(cur.x, x);
    if (POST) {
      float u[kE];
      widen(cur.u, u);
      standardise<G, VEC, false>(u, u, g, p);
      if (gated) {
        float q[kE];
        widen(cur.gate, q);
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = fmaf(fmaf(u[e], g1[e], b1[e]), sigmoid(q[e]), x[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] += fmaf(u[e], g1[e], b1[e]);
      }
      if (live && g.act)
        Store<TS, VEC>::put(row_ptr(p.x1, r, flat), g.lane, g.lanes, C, x);
    }
    if (PRE) {
      standardise<G, VEC, false>(x, x, g, p);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] = fmaf(x[e], g2[e], b2[e]);
      if (live && g.act)
        Store<TI, VEC>::put(row_ptr(p.y, r, flat), g.lane, g.lanes, C, x);
    }
    cur = nxt;
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// GROUPED: gate rows shared by consecutive rows, whose gradients are summed.
template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE, bool GROUPED>
__global__ void __launch_bounds__(G == 0 ? 512 : kThreads)
    k_block_norm_bwd(const __grid_constant__ Params p) {
  __shared__ float2 sums[8][2 * kMaxWarps];
  extern __shared__ float red[];  // [slots][lanes * 8]
  Group g = make_group<G, VEC>(p, sums);
  const int C = p.C;
  const bool flat = p.rows_of.flat;
  const bool gated = POST && (GROUPED || p.gate.p != nullptr);

  float sc[kE], g1[kE], b1[kE], g2[kE];
  if (POST) {
    param<VEC>(p.scale, 1.f, g.lane, g.lanes, C, sc);
    param<VEC>(p.gamma_post, 1.f, g.lane, g.lanes, C, g1);
    param<VEC>(p.beta_post, 0.f, g.lane, g.lanes, C, b1);
  }
  if (PRE) param<VEC>(p.gamma_pre, 1.f, g.lane, g.lanes, C, g2);

  float acc[5][kE];
#pragma unroll
  for (int k = 0; k < 5; ++k)
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[k][e] = 0.f;
  float q[kE], dg[kE];  // sigmoid(gate) and the gate's gradient
#pragma unroll
  for (int e = 0; e < kE; ++e) q[e] = 1.f;

  struct In {
    Raw<TS, VEC> x1, dx1;
    Raw<TI, VEC> u, gate, dy;
  };
  auto fetch = [&](In& in, uint32_t row) {
    const RowPos r = row_pos(p.rows_of, row);
    if (!g.act) return;
    if (p.dx1.p) load(in.dx1, row_ptr(p.dx1, r, flat), g.lane, g.lanes, C);
    if (PRE) {
      load(in.x1, row_ptr(p.x, r, flat), g.lane, g.lanes, C);
      load(in.dy, row_ptr(p.dy, r, flat), g.lane, g.lanes, C);
    }
    if (POST) {
      load(in.u, row_ptr(p.u, r, flat), g.lane, g.lanes, C);
      if (!GROUPED && gated) load(in.gate, row_ptr(p.gate, r, flat), g.lane, g.lanes, C);
    }
  };

  // one row's gradients; a group without a row (live = false) only takes part
  // in the sums, on the zeros that it holds
  auto work = [&](In& in, uint32_t row, bool live) {
    const RowPos r = row_pos(p.rows_of, live ? row : 0);
    if (!live) in = In{};
    float D[kE], u[kE], h[kE];
    widen(in.dx1, D);
    float2 rstd;
    if (POST) widen(in.u, u);
    if (PRE) {
      widen(in.x1, h);
      rstd = standardise<G, VEC, POST>(h, u, g, p);
    } else {
      rstd = standardise<G, VEC, false>(u, u, g, p);
      rstd.y = rstd.x;
    }
    if (PRE) {
      float dy[kE];
      widen(in.dy, dy);
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        acc[3][e] = fmaf(dy[e], h[e], acc[3][e]);
        acc[4][e] += dy[e];
        dy[e] *= g2[e];
        s.x += dy[e];
        s.y = fmaf(dy[e], h[e], s.y);
      }
      if (!g.act) s = make_float2(0.f, 0.f);
      s = group_sum<G>(s, g.sum);
      const float m0 = p.rms ? 0.f : s.x * p.inv_c, m1 = s.y * p.inv_c;
#pragma unroll
      for (int e = 0; e < kE; ++e)
        D[e] = fmaf(rstd.x, fmaf(-m1, h[e], dy[e] - m0), D[e]);
      if (live && g.act)
        Store<TS, VEC>::put(row_ptr(p.dx, r, flat), g.lane, g.lanes, C, D);
    }
    if (POST) {
      if (!GROUPED && gated) {
        float v[kE];
        widen(in.gate, v);
#pragma unroll
        for (int e = 0; e < kE; ++e) q[e] = sigmoid(v[e]);
      }
      float b[kE];
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float w = fmaf(u[e], g1[e], b1[e]);
        const float dq = D[e] * q[e];
        acc[0][e] = fmaf(dq, w, acc[0][e]);
        const float en = dq * sc[e];
        if (GROUPED)
          dg[e] = fmaf(en, w, dg[e]);  // (1 - q) is applied once, at the end
        else
          dg[e] = en * w * (1.f - q[e]);
        acc[1][e] = fmaf(en, u[e], acc[1][e]);
        acc[2][e] += en;
        b[e] = en * g1[e];
        s.x += b[e];
        s.y = fmaf(b[e], u[e], s.y);
      }
      if (!g.act) s = make_float2(0.f, 0.f);
      s = group_sum<G>(s, g.sum);
      const float m0 = p.rms ? 0.f : s.x * p.inv_c, m1 = s.y * p.inv_c;
#pragma unroll
      for (int e = 0; e < kE; ++e) b[e] = rstd.y * fmaf(-m1, u[e], b[e] - m0);
      if (live && g.act) {
        Store<TI, VEC>::put(row_ptr(p.du, r, flat), g.lane, g.lanes, C, b);
        if (!GROUPED && gated)
          Store<TI, VEC>::put(row_ptr(p.dgate, r, flat), g.lane, g.lanes, C, dg);
      }
    }
  };

  if (!GROUPED) {
    const uint32_t step = gridDim.x * g.slots;
    uint32_t first = blockIdx.x * g.slots;
    In cur{}, nxt{};
    if (first + g.slot < p.rows) fetch(cur, first + g.slot);
    for (; first < p.rows; first += step) {
      const uint32_t row = first + g.slot;
      if (row + step < p.rows) fetch(nxt, row + step);
      work(cur, row, row < p.rows);
      cur = nxt;
    }
  } else {
    // items of consecutive rows under one gate row: spread over the CTA's
    // groups, or walked by one group each
    const uint32_t per_cta = p.by_cta ? 1u : (uint32_t)g.slots;
    const uint32_t hop = p.by_cta ? (uint32_t)g.slots : 1u;
    for (uint32_t first = blockIdx.x * per_cta; first < p.items; first += gridDim.x * per_cta) {
      const uint32_t item = p.by_cta ? first : first + g.slot;
      const bool mine = item < p.items;
      const uint32_t gate_row = mine ? item / p.segs : 0;
      const uint32_t seg = mine ? item - gate_row * p.segs : 0;
      const uint32_t begin = gate_row * p.share + seg * p.seg_rows;
      const uint32_t end = mine ? min(gate_row * p.share + p.share, begin + p.seg_rows) : begin;
      const RowPos at = row_pos(p.rows_of, gate_row * p.share);
      Raw<TI, VEC> raw{};
      if (g.act) load(raw, row_ptr(p.gate, at, flat), g.lane, g.lanes, C);
      widen(raw, q);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        q[e] = sigmoid(q[e]);
        dg[e] = 0.f;
      }
      uint32_t row = begin + (p.by_cta ? (uint32_t)g.slot : 0u);
      In cur{}, nxt{};
      if (row < end) fetch(cur, row);
      // the same number of turns for every group of the CTA
      for (uint32_t t = 0; t < p.seg_rows; t += hop, row += hop) {
        if (row + hop < end) fetch(nxt, row + hop);
        work(cur, row, row < end);
        cur = nxt;
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) dg[e] *= 1.f - q[e];
      if (p.by_cta && g.slots > 1) {
        const int width = g.lanes * kE;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kE; ++e)
          red[g.slot * width + channel<VEC>(g.lane, g.lanes, e)] = dg[e];
        __syncthreads();
        if (g.slot == 0) {
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            float s = 0.f;
            for (int i = 0; i < g.slots; ++i) s += red[i * width + channel<VEC>(g.lane, g.lanes, e)];
            dg[e] = s;
          }
        }
      }
      if (mine && g.act && (!p.by_cta || g.slot == 0)) {
        if (p.segs == 1)
          Store<TI, VEC>::put(row_ptr(p.dgate, at, flat), g.lane, g.lanes, C, dg);
        else
          Store<float, VEC>::put(reinterpret_cast<char*>(p.gate_part + (size_t)item * C), g.lane,
                                 g.lanes, C, dg);
      }
    }
  }

  // the CTA's sums of the parameter gradients, group by group in order
  const int width = g.lanes * kE;
#pragma unroll
  for (int k = POST ? 0 : 3; k < (PRE ? 5 : 3); ++k) {
    if (p.out[k] == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kE; ++e)
      red[g.slot * width + channel<VEC>(g.lane, g.lanes, e)] = acc[k][e];
    __syncthreads();
    float* dst = gridDim.x == 1 ? p.out[k] : p.part + ((size_t)blockIdx.x * 5 + k) * C;
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float s = 0.f;
      for (int i = 0; i < g.slots; ++i) s += red[i * width + c];
      dst[c] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Resident CTAs of a kernel per SM times the SMs, looked up once per device.
template <typename K>
cudaError_t resident_ctas(K kernel, int threads, size_t smem, std::atomic<int> (&cache)[64][17],
                          int key, int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64) *n = cache[dev][key].load(std::memory_order_relaxed);
  else *n = 0;
  if (*n > 0) return cudaSuccess;
  int sms = 0, per = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *n = std::max(1, sms) * std::max(1, per);
  if (dev >= 0 && dev < 64) cache[dev][key].store(*n, std::memory_order_relaxed);
  return cudaSuccess;
}

// The launch's row space.  Axes along which the gate does not move come last,
// the others by the stride of the first operand given; neighbouring axes that every
// operand walks as one become one (never across the border between the two
// kinds, which is where a gate row's rows begin).
struct Axes {
  uint32_t n[3];
  int64_t s[3][10];
  uint32_t share;
};
inline Axes order_axes(const int (&n)[3], const RowOperand* const* ops, int count, int gate_at) {
  struct Axis {
    uint32_t n;
    int64_t s[10];
    bool shared;
  };
  Axis ax[3];
  int k = 0;
  for (int d = 0; d < 3; ++d) {
    if (n[d] == 1) continue;
    ax[k].n = (uint32_t)n[d];
    for (int i = 0; i < count; ++i) ax[k].s[i] = ops[i]->p ? ops[i]->s[d] : 0;
    ax[k].shared = gate_at >= 0 && ax[k].s[gate_at] == 0;
    ++k;
  }
  int lead = 0;
  while (lead + 1 < count && !ops[lead]->p) ++lead;
  std::stable_sort(ax, ax + k, [lead](const Axis& a, const Axis& b) {
    if (a.shared != b.shared) return !a.shared;
    return a.s[lead] > b.s[lead];
  });
  Axes out{};
  out.share = 1;
  for (int d = 0; d < k; ++d)
    if (ax[d].shared) out.share *= ax[d].n;
  int m = 0;
  for (int d = 0; d < k; ++d) {
    bool join = m > 0 && ax[m - 1].shared == ax[d].shared;
    for (int i = 0; join && i < count; ++i)
      if (ops[i]->p) join = ax[m - 1].s[i] == ax[d].s[i] * (int64_t)ax[d].n;
    if (join) {
      const uint32_t outer = ax[m - 1].n;
      ax[m - 1] = ax[d];
      ax[m - 1].n = outer * ax[d].n;
    } else {
      ax[m++] = ax[d];
    }
  }
  for (int d = 0; d < 3; ++d) {  // right-aligned: the innermost axis is [2]
    const int from = d - (3 - m);
    out.n[d] = from >= 0 ? ax[from].n : 1u;
    for (int i = 0; i < count; ++i) out.s[d][i] = from >= 0 ? ax[from].s[i] : 0;
  }
  return out;
}

struct Plan {
  Params p;
  int g;        // lanes of a row's group: 8, 16, 32, or 0 for several warps
  bool vec;
  int threads, slots;
};

// Sizes and operands, for both directions: `ops` go to `dst` (parts of pl.p),
// their element sizes in `esize`.
inline void make_plan(const BlockNormCall& c, const RowOperand* const* ops, Operand* const* dst,
                      const int* esize, int count, int gate_at, Plan& pl) {
  Params& p = pl.p;
  const Axes ax = order_axes(c.n, ops, count, gate_at);
  p.rows = ax.n[0] * ax.n[1] * ax.n[2];
  p.rows_of.d2 = fast_div(ax.n[2]);
  p.rows_of.d1 = fast_div(ax.n[1]);
  p.rows_of.flat = ax.n[0] == 1 && ax.n[1] == 1;
  p.share = ax.share;
  pl.vec = c.C % kE == 0;
  for (int i = 0; i < count; ++i) {
    Operand& o = *dst[i];
    o.p = static_cast<char*>(ops[i]->p);
    if (!o.p) continue;
    o.s0 = ax.s[0][i] * esize[i];
    o.s1 = ax.s[1][i] * esize[i];
    o.s2 = ax.s[2][i] * esize[i];
    if (reinterpret_cast<uintptr_t>(o.p) % 16 || o.s0 % 16 || o.s1 % 16 || o.s2 % 16) pl.vec = false;
  }
  p.C = c.C;
  p.rms = c.rms;
  p.eps = c.eps;
  p.inv_c = 1.0f / (float)c.C;
  p.scale = c.scale;
  p.gamma_post = c.gamma_post;
  p.beta_post = c.beta_post;
  p.gamma_pre = c.gamma_pre;
  p.beta_pre = c.beta_pre;
  const int need = (c.C + kE - 1) / kE;  // threads of a row
  if (need <= 32) {
    pl.g = pl.vec ? (need <= 8 ? 8 : need <= 16 ? 16 : 32) : 32;
    p.lanes = pl.g;
    pl.threads = kThreads;
  } else {
    pl.g = 0;
    const int warps = (need + 31) / 32;
    p.lanes = warps * 32;
    pl.threads = p.lanes * std::max(1, kThreads / 32 / warps);
  }
  pl.slots = pl.threads / p.lanes;
}

// Sums of the CTAs' partial sums: one block per 32 columns of one of the five
// parameter gradients or of one gate row, 8 warps taking every 8th partial.
template <typename TI>
__global__ void __launch_bounds__(256) k_block_norm_reduce(const __grid_constant__ Params p,
                                                           int ctas, int param_blocks) {
  __shared__ float red[8][32];
  const int per = (p.C + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blk = blockIdx.x;
  const bool is_param = blk < param_blocks;
  const int what = (is_param ? blk : blk - param_blocks) / per;
  const int c = ((is_param ? blk : blk - param_blocks) - what * per) * 32 + lane;
  if (is_param && p.out[what] == nullptr) return;
  const int depth = is_param ? ctas : (int)p.segs;
  const float* src = is_param ? p.part + (size_t)what * p.C : p.gate_part + (size_t)what * p.segs * p.C;
  const size_t stride = (size_t)p.C * (is_param ? 5 : 1);
  float s = 0.f;
  if (c < p.C) {
#pragma unroll 4
    for (int i = warp; i < depth; i += 8) s += src[i * stride + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    if (is_param) {
      p.out[what][c] = s;
    } else {
      char* row = row_ptr(p.dgate, row_pos(p.rows_of, (uint32_t)what * p.share), p.rows_of.flat);
      reinterpret_cast<TI*>(row)[c] = static_cast<TI>(s);
    }
  }
}

template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE>
cudaError_t launch_fwd(const Plan& pl, cudaStream_t st) {
  static std::atomic<int> cache[64][17];
  auto kern = k_block_norm_fwd<TS, TI, G, VEC, POST, PRE>;
  int ctas = 0;
  cudaError_t e = resident_ctas(kern, pl.threads, 0, cache, pl.threads / 32, &ctas);
  if (e != cudaSuccess) return e;
  const unsigned need = (pl.p.rows + pl.slots - 1) / pl.slots;
  kern<<<std::min<unsigned>(need, (unsigned)ctas), pl.threads, 0, st>>>(pl.p);
  return cudaGetLastError();
}

template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE, bool GROUPED>
cudaError_t launch_bwd(Plan pl, float* ws, cudaStream_t st) {
  static std::atomic<int> cache[64][17];
  auto kern = k_block_norm_bwd<TS, TI, G, VEC, POST, PRE, GROUPED>;
  Params& p = pl.p;
  const size_t smem = (size_t)pl.slots * p.lanes * kE * sizeof(float);
  int ctas = 0;
  cudaError_t e = resident_ctas(kern, pl.threads, smem, cache, pl.threads / 32, &ctas);
  if (e != cudaSuccess) return e;
  ctas = std::min(ctas, kNormMaxCtas);
  unsigned need = (p.rows + pl.slots - 1) / pl.slots;
  if (GROUPED) {
    // A gate row's rows are walked by one group where they are fewer than the
    // CTA's groups (spreading them would leave groups idle), else spread over
    // a CTA, in as many items per gate row as give every CTA one.
    const uint32_t gates = p.rows / p.share;
    p.by_cta = p.share >= (uint32_t)pl.slots;
    p.segs = 1;
    p.seg_rows = p.share;
    if (p.by_cta && gates < (uint32_t)ctas) {
      const uint32_t want = ((uint32_t)ctas + gates - 1) / gates;
      p.seg_rows = std::max<uint32_t>(pl.slots, (p.share + want - 1) / want);
      p.seg_rows = (p.seg_rows + pl.slots - 1) / pl.slots * pl.slots;
      p.segs = (p.share + p.seg_rows - 1) / p.seg_rows;
    }
    p.items = gates * p.segs;
    need = p.by_cta ? p.items : (p.items + pl.slots - 1) / pl.slots;
  }
  const unsigned grid = std::min<unsigned>(need, (unsigned)ctas);
  p.part = ws;
  p.gate_part = ws + (size_t)kNormMaxCtas * 5 * p.C;
  kern<<<grid, pl.threads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per = (p.C + 31) / 32;
  bool any = false;
  for (int k = 0; k < 5; ++k) any = any || p.out[k] != nullptr;
  const int param_blocks = any && grid > 1 ? 5 * per : 0;
  const int gate_blocks = GROUPED && p.segs > 1 ? (int)(p.rows / p.share) * per : 0;
  if (param_blocks + gate_blocks > 0) {
    k_block_norm_reduce<TI><<<param_blocks + gate_blocks, 256, 0, st>>>(p, (int)grid, param_blocks);
    e = cudaGetLastError();
  }
  return e;
}

template <typename TS, typename TI, bool POST, bool PRE>
cudaError_t dispatch_fwd(const Plan& pl, cudaStream_t st) {
  if (pl.vec) {
    switch (pl.g) {
      case 8: return launch_fwd<TS, TI, 8, true, POST, PRE>(pl, st);
      case 16: return launch_fwd<TS, TI, 16, true, POST, PRE>(pl, st);
      case 32: return launch_fwd<TS, TI, 32, true, POST, PRE>(pl, st);
      default: return launch_fwd<TS, TI, 0, true, POST, PRE>(pl, st);
    }
  }
  return pl.g ? launch_fwd<TS, TI, 32, false, POST, PRE>(pl, st)
              : launch_fwd<TS, TI, 0, false, POST, PRE>(pl, st);
}

template <typename TS, typename TI, bool POST, bool PRE, bool GROUPED>
cudaError_t dispatch_bwd(const Plan& pl, float* ws, cudaStream_t st) {
  if (pl.vec) {
    switch (pl.g) {
      case 8: return launch_bwd<TS, TI, 8, true, POST, PRE, GROUPED>(pl, ws, st);
      case 16: return launch_bwd<TS, TI, 16, true, POST, PRE, GROUPED>(pl, ws, st);
      case 32: return launch_bwd<TS, TI, 32, true, POST, PRE, GROUPED>(pl, ws, st);
      default: return launch_bwd<TS, TI, 0, true, POST, PRE, GROUPED>(pl, ws, st);
    }
  }
  return pl.g ? launch_bwd<TS, TI, 32, false, POST, PRE, GROUPED>(pl, ws, st)
              : launch_bwd<TS, TI, 0, false, POST, PRE, GROUPED>(pl, ws, st);
}

template <typename TS, typename TI>
cudaError_t run_fwd(const BlockNormCall& c, cudaStream_t st) {
  constexpr int S = sizeof(TS), I = sizeof(TI);
  Plan pl{};
  Params& p = pl.p;
  const RowOperand* ops[] = {&c.x, &c.u, &c.gate, &c.x1, &c.y};
  Operand* dst[] = {&p.x, &p.u, &p.gate, &p.x1, &p.y};
  const int es[] = {S, I, I, S, I};
  make_plan(c, ops, dst, es, 5, -1, pl);
  if (c.u.p && c.y.p) return dispatch_fwd<TS, TI, true, true>(pl, st);
  if (c.u.p) return dispatch_fwd<TS, TI, true, false>(pl, st);
  return dispatch_fwd<TS, TI, false, true>(pl, st);
}

template <typename TS, typename TI>
cudaError_t run_bwd(const BlockNormCall& c, cudaStream_t st) {
  constexpr int S = sizeof(TS), I = sizeof(TI);
  Plan pl{};
  Params& p = pl.p;
  const RowOperand* ops[] = {&c.dx1, &c.x, &c.u, &c.gate, &c.dy, &c.dx, &c.du, &c.dgate};
  Operand* dst[] = {&p.dx1, &p.x, &p.u, &p.gate, &p.dy, &p.dx, &p.du, &p.dgate};
  const int es[] = {S, S, I, I, I, S, I, I};
  make_plan(c, ops, dst, es, 8, c.gate.p ? 3 : -1, pl);
  p.out[0] = c.dscale;
  p.out[1] = c.dgamma_post;
  p.out[2] = c.dbeta_post;
  p.out[3] = c.dgamma_pre;
  p.out[4] = c.dbeta_pre;
  const bool grouped = c.gate.p && p.share > 1;
  if (c.u.p && c.dy.p)
    return grouped ? dispatch_bwd<TS, TI, true, true, true>(pl, c.ws, st)
                   : dispatch_bwd<TS, TI, true, true, false>(pl, c.ws, st);
  if (c.u.p)
    return grouped ? dispatch_bwd<TS, TI, true, false, true>(pl, c.ws, st)
                   : dispatch_bwd<TS, TI, true, false, false>(pl, c.ws, st);
  return dispatch_bwd<TS, TI, false, true, false>(pl, c.ws, st);
}

}  // namespace norm
}  // namespace evo
