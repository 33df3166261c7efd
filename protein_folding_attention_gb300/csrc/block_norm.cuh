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
//                              (1 - q = e^-gate q, without cancellation)
//   dgamma_post = sum e k      dbeta_post = sum e             b = e gamma_post
//   du = rstd (b - mean(b) - k mean(b k))
//   dgamma_pre = sum dy h      dbeta_pre = sum dy
//
// With A = sum D q k and B = sum D q, kept per channel, dscale is
// gamma_post A + beta_post B, dgamma_post is scale A and dbeta_post scale B.
// (rms: mean = 0 and no mean(a), mean(b) terms.)  Everything is held in fp32;
// each stored tensor is rounded once.  Bound by HBM: 10 bytes per element
// forward and 16 backward in bf16, against about 20 and 50 fp32 operations.
//
// Layout: a row belongs to a group of G threads, 8 channels each, so that a
// bf16 row is one 16-byte access per thread and its values stay in registers
// from load to store.  G = 8, 16 or 32 lanes of a warp up to C = 256, or for
// narrow bf16 rows as many lanes as they have parts (sums by
// shuffles); a warp with two such parts per lane up to C = 512; above that
// several warps (sums by shuffles, then through shared memory with one named
// barrier per sum).  The forward's CTAs are many and short, the backward's
// persistent (launch_fwd, launch_bwd).  A thread
// copies its own channels of the coming rows into a ring in shared memory
// (cp.async, no registers held meanwhile, no barrier: it reads only what it
// copied), and keeps the parameter gradients of its channels over all its rows
// in registers.  The CTAs' sums go to the workspace and a second kernel adds
// them in a fixed order: repeated calls give the same bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block_norm.h"
#include "common.cuh"
#include "launch.cuh"

namespace evo {
namespace norm {
// (each including file has its own copies: a function's static data must not
// be shared with another copy of this library in the process)
namespace {

constexpr int kSums = 4;          // vectors that the backward sums over rows
constexpr int kE = 8;             // channels of a part: what a thread has of a row, or half of it
constexpr int kThreads = 256;     // threads of a CTA where a row takes at most 8 warps
constexpr int kMaxThreads = 512;  // ... 16 warps (C = 4096)

// How a row is laid over threads: 8, 16 or 32 lanes of a warp, or as many as it
// has parts; a whole warp with two parts per lane; up to 8 warps, with one part or two; or any number
// of warps, one part each (rows that cannot be copied 16 bytes at a time).
constexpr int kTwice = 64, kWarps = 0, kPlain = -1, kWarpsTwice = -2, kPacked = 10;
constexpr bool warps_of(int G) { return G <= 0; }
constexpr int width_of(int G) { return G <= 0 || G > 32 ? 32 : G; }  // lanes of a warp that share a row
constexpr int parts_of(int G) { return G == kTwice || G == kWarpsTwice ? 2 : 1; }
constexpr bool ring_of(int G, bool vec) { return vec && G != kPlain; }
constexpr int threads_of(int G) { return G == kPlain ? kMaxThreads : G == kTwice ? kThreads / 2 : kThreads; }

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
__device__ __forceinline__ char* row_ptr(const Operand& o, const RowPos& r, const Rows& R) {
  char* p = o.p + r.i2 * o.s2;
  if (!R.flat) p += r.i1 * o.s1 + r.i0 * o.s0;
  return p;
}

struct Params {
  Rows rows_of;   // row axes of every operand
  Rows gate_of;   // axes of the gate's own rows, where rows share them
  FastDiv by_share;
  uint32_t rows;
  uint32_t turns;  // forward: rows of each group of a CTA
  uint32_t stride_s, stride_i;  // DENSE: bytes between rows of the stream's and the block's operands
  int C;
  int lanes;      // threads of a row's group (a multiple of 32 where it spans warps)
  bool rms;
  bool wide_params;  // the parameter vectors are 16-byte aligned
  float eps, inv_c;
  Operand x, u, gate, x1, y, dx1, dy, dx, du, dgate;
  const float *scale, *gamma_post, *beta_post, *gamma_pre, *beta_pre;
  float *dscale, *dgamma_post, *dbeta_post, *dgamma_pre, *dbeta_pre;
  bool wanted[2];  // any gradient of the post-norm's, of the pre-norm's parameters
  float* part;     // [CTAs][kSums][C]
  // a gate row shared by `share` consecutive rows: `segs` items of at most
  // `seg_rows` rows each per gate row
  uint32_t share, segs, seg_rows, items;
  bool by_cta;       // an item's rows are spread over the CTA (else one group walks them)
  bool in_step;      // the CTA's warps meet at every turn (see launch_bwd)
  float* gate_part;  // [items][C] where segs > 1
};

// Where a row lies.  DENSE: every operand has one row axis, with one stride
// for all of the stream's operands and one for all of the block's (the usual
// case; a third of the address arithmetic).
template <bool DENSE>
struct At {
  RowPos r;
  uint64_t s, i;
  __device__ __forceinline__ At(const Params& p, uint32_t row) {
    if constexpr (DENSE) {
      s = (uint64_t)row * p.stride_s;
      i = (uint64_t)row * p.stride_i;
    } else {
      r = row_pos(p.rows_of, row);
    }
  }
  __device__ __forceinline__ char* stream(const Params& p, const Operand& o) const {
    if constexpr (DENSE) return o.p + s;
    else return row_ptr(o, r, p.rows_of);
  }
  __device__ __forceinline__ char* block(const Params& p, const Operand& o) const {
    if constexpr (DENSE) return o.p + i;
    else return row_ptr(o, r, p.rows_of);
  }
};

// ---------------------------------------------------------------------------
// a thread's channels of a row, in pairs
// ---------------------------------------------------------------------------
// Which channels: 8 in a row (16 bytes of bf16); where the stream is fp32 two
// runs of 4, the second behind the first runs of all threads that share a row
// (of a warp, where a row spans several), so that neighbouring threads touch
// neighbouring 16 bytes; or, where C is no multiple of 8 or a row is not
// 16-byte aligned, every lanes-th channel, one element per access.
enum Layout { kRun, kSplit, kSingle };
template <typename TS, bool VEC>
constexpr Layout layout_of() { return !VEC ? kSingle : sizeof(TS) == 2 ? kRun : kSplit; }

template <int Q>
struct Vec {
  static constexpr int E = kE * Q, P = E / 2;
  float2 p[P];
  __device__ __forceinline__ float& operator[](int e) { return e & 1 ? p[e >> 1].y : p[e >> 1].x; }
  __device__ __forceinline__ float operator[](int e) const { return e & 1 ? p[e >> 1].y : p[e >> 1].x; }
};
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
template <int Q>
__device__ __forceinline__ float sum(const Vec<Q>& v) {
  float2 s = add2(add2(v.p[0], v.p[1]), add2(v.p[2], v.p[3]));
  if constexpr (Q == 2) s = add2(s, add2(add2(v.p[4], v.p[5]), add2(v.p[6], v.p[7])));
  return s.x + s.y;
}
template <int Q>
__device__ __forceinline__ float dot(const Vec<Q>& a, const Vec<Q>& b) {
  float2 s = mul2(a.p[1], b.p[1]), t = mul2(a.p[3], b.p[3]);
  s = fma2(a.p[0], b.p[0], s);
  t = fma2(a.p[2], b.p[2], t);
#pragma unroll
  for (int k = 4; k < Vec<Q>::P; k += 2) {
    s = fma2(a.p[k], b.p[k], s);
    t = fma2(a.p[k + 1], b.p[k + 1], t);
  }
  const float2 r = add2(s, t);
  return r.x + r.y;
}

// What a thread knows of its group.
struct Group {
  int lane, lanes;  // place in the row's group
  int slot, slots;  // the group's place in the CTA
  int c0, c1;       // first channels of its two runs of 4
  int l, first;     // place in its warp's part of the group, and that part's first thread
  int base;         // that part's first channel
  bool act;         // it has channels
  float2* buf;      // sums across warps, [2][kMaxWarps]
  int turn;
};
template <Layout L, int G>
__device__ __forceinline__ int channel(const Group& g, int e) {
  if (L == kSingle) return e * g.lanes + g.lane;
  const int f = e % kE;
  return (f < 4 ? g.c0 + f : g.c1 + f - 4) + e / kE * (kE * width_of(G));
}
// First channel of a run of 4.
template <int G>
__device__ __forceinline__ int run(const Group& g, int h) {
  return (h & 1 ? g.c1 : g.c0) + h / 2 * (kE * width_of(G));
}

template <int Q>
__device__ __forceinline__ void put_run(Vec<Q>& v, int h, float4 q) {
  v.p[2 * h] = make_float2(q.x, q.y);
  v.p[2 * h + 1] = make_float2(q.z, q.w);
}
template <int Q>
__device__ __forceinline__ void put_run(Vec<Q>& v, int h, uint2 q) {
  v.p[2 * h] = make_float2(bf16lo(q.x), bf16hi(q.x));
  v.p[2 * h + 1] = make_float2(bf16lo(q.y), bf16hi(q.y));
}
template <int Q>
__device__ __forceinline__ void put_part(Vec<Q>& v, int k, uint4 q) {
  put_run(v, 2 * k, make_uint2(q.x, q.y));
  put_run(v, 2 * k + 1, make_uint2(q.z, q.w));
}
template <int Q>
__device__ __forceinline__ uint2 narrow(const Vec<Q>& v, int h) {
  const float2 a = v.p[2 * h], b = v.p[2 * h + 1];
  return make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
}

template <typename T, Layout L, int G>
__device__ __forceinline__ Vec<parts_of(G)> load(const char* row, const Group& g, int C) {
  constexpr int Q = parts_of(G);
  Vec<Q> v{};
  const T* p = reinterpret_cast<const T*>(row);
  if constexpr (L == kSingle) {
#pragma unroll
    for (int e = 0; e < v.E; ++e) {
      const int c = channel<L, G>(g, e);
      if (c < C) v[e] = static_cast<float>(p[c]);
    }
  } else if constexpr (L == kRun && sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const int c = run<G>(g, 2 * k);
      if (c < C) put_part(v, k, *reinterpret_cast<const uint4*>(p + c));
    }
  } else {
    using Run = typename std::conditional<sizeof(T) == 2, uint2, float4>::type;
#pragma unroll
    for (int h = 0; h < 2 * Q; ++h) {
      const int c = run<G>(g, h);
      if (c < C) put_run(v, h, *reinterpret_cast<const Run*>(p + c));
    }
  }
  return v;
}

// Writes a thread's channels where `live`.
template <typename T, Layout L, int G>
__device__ __forceinline__ void store(bool live, char* row, const Group& g, int C, const Vec<parts_of(G)>& v) {
  constexpr int Q = parts_of(G);
  T* p = reinterpret_cast<T*>(row);
  if constexpr (L == kSingle) {
#pragma unroll
    for (int e = 0; e < v.E; ++e) {
      const int c = channel<L, G>(g, e);
      if (live && c < C) p[c] = static_cast<T>(v[e]);
    }
  } else if constexpr (L == kRun && sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const int c = run<G>(g, 2 * k);
      const uint2 a = narrow(v, 2 * k), b = narrow(v, 2 * k + 1);
      if (live && c < C) *reinterpret_cast<uint4*>(p + c) = make_uint4(a.x, a.y, b.x, b.y);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2 * Q; ++h) {
      const int c = run<G>(g, h);
      if (!live || c >= C) continue;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(p + c) = narrow(v, h);
      else
        *reinterpret_cast<float4*>(p + c) =
            make_float4(v.p[2 * h].x, v.p[2 * h].y, v.p[2 * h + 1].x, v.p[2 * h + 1].y);
    }
  }
}

// A thread's channels of a parameter vector (`absent` without one).
template <Layout L, int G>
__device__ __forceinline__ Vec<parts_of(G)> param(const float* p, float absent, const Group& g, int C, bool wide) {
  Vec<parts_of(G)> v{};
  if (L != kSingle && wide && p) {
#pragma unroll
    for (int h = 0; h < 2 * parts_of(G); ++h) {
      const int c = run<G>(g, h);
      if (c < C) put_run(v, h, *reinterpret_cast<const float4*>(p + c));
    }
    return v;
  }
#pragma unroll
  for (int e = 0; e < v.E; ++e) {
    const int c = channel<L, G>(g, e);
    v[e] = c < C ? (p ? p[c] : absent) : 0.f;
  }
  return v;
}

// The ring: copies of 16 bytes, consecutive threads to consecutive places.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  // (bytes = 0 reads nothing and fills with zeros)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 16-byte units of a part
template <typename T>
constexpr int units() { return kE * (int)sizeof(T) / 16; }
template <typename T, int G>
__host__ __device__ constexpr uint32_t ring_bytes(uint32_t threads) {
  return threads * 16 * units<T>() * parts_of(G);
}

// The lanes of a warp that share a row copy it part by part.  A thread reads
// what it copied itself, but for the bf16 rows of kSplit, of which it copies 8
// channels in a row and reads its two runs of 4.
template <typename T, Layout L, int G>
__device__ __forceinline__ void ring_put(uint32_t stage, const char* row, const Group& g, int C, bool live) {
  constexpr int W = width_of(G), Q = parts_of(G);
  const uint32_t to = stage + g.first * (16 * units<T>() * Q) + g.l * 16;
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    if constexpr (sizeof(T) == 2) {
      const int c = g.base + kE * (g.l + k * W);
      const uint32_t bytes = live && c < C ? 16u : 0u;
      copy16(to + k * (W * 16), row + (bytes ? c * 2 : 0), bytes);
    } else {
      const int a = run<G>(g, 2 * k), b = run<G>(g, 2 * k + 1);
      const uint32_t na = live && a < C ? 16u : 0u, nb = live && b < C ? 16u : 0u;
      copy16(to + k * (W * 32), row + (na ? a * 4 : 0), na);
      copy16(to + k * (W * 32) + W * 16, row + (nb ? b * 4 : 0), nb);
    }
  }
}
template <typename T, Layout L, int G>
__device__ __forceinline__ Vec<parts_of(G)> ring_get(const char* stage, const Group& g) {
  constexpr int W = width_of(G), Q = parts_of(G);
  Vec<Q> v;
  const char* from = stage + g.first * (16 * units<T>() * Q);
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    if constexpr (sizeof(T) == 2 && L == kRun) {
      put_part(v, k, *reinterpret_cast<const uint4*>(from + g.l * 16 + k * (W * 16)));
    } else if constexpr (sizeof(T) == 2) {
      const char* at = from + g.l * 8 + k * (W * 16);
      put_run(v, 2 * k, *reinterpret_cast<const uint2*>(at));
      put_run(v, 2 * k + 1, *reinterpret_cast<const uint2*>(at + W * 8));
    } else {
      const char* at = from + g.l * 16 + k * (W * 32);
      put_run(v, 2 * k, *reinterpret_cast<const float4*>(at));
      put_run(v, 2 * k + 1, *reinterpret_cast<const float4*>(at + W * 16));
    }
  }
  return v;
}

// Rows that cannot be copied one by one in 16-byte units (C no multiple of 8)
// but lie one behind the other from a 16-byte aligned address on: the rows of
// a CTA's turn are then copied as one piece, from the 16 bytes that its first
// byte lies in to its last byte.  (The up to 14 bytes before the first are the
// row's before it.)
__host__ __device__ constexpr uint32_t chunk_size(uint32_t elements, uint32_t esize) {
  return (elements * esize + 15) / 16 * 16 + 16;
}
__device__ __forceinline__ void chunk_put(uint32_t to, const char* src, uint32_t bytes, uint32_t shift) {
  src -= shift;
  bytes += shift;
  for (uint32_t at = threadIdx.x * 16; at < bytes; at += blockDim.x * 16)
    copy16(to + at, src + at, min(16u, bytes - at));
}

// ---------------------------------------------------------------------------
// sums over a row's group
// ---------------------------------------------------------------------------
// G lanes of a warp, or several warps: then every warp leaves its sum
// in shared memory and reads all of them behind one barrier.  Two buffers take
// turns, so that a sum's values are read before the barrier that precedes
// their buffer's next use.
constexpr int kMaxWarps = 16;
__device__ __forceinline__ float2 across_warps(float2 v, Group& g) {
  float2* b = g.buf + (g.turn ? kMaxWarps : 0);
  g.turn ^= 1;
  const int warps = g.lanes >> 5;
  if ((threadIdx.x & 31) == 0) b[g.lane >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + g.slot), "r"(g.lanes) : "memory");
  v = make_float2(0.f, 0.f);
  for (int i = 0; i < warps; ++i) v = add2(v, b[i]);
  return v;
}
// n <= 16 lanes, any number: lane l takes lane l + o, then all take the first's.
__device__ __forceinline__ float packed_sum(float v, const Group& g) {
  auto take = [&](int o) {
    const float t = __shfl_down_sync(0xffffffffu, v, o);
    if (g.l + o < g.lanes) v += t;
  };
  if (g.lanes > 8) take(8);
  take(4);
  take(2);
  take(1);
  return __shfl_sync(0xffffffffu, v, (int)(threadIdx.x & 31) - g.l);
}
template <int G>
__device__ __forceinline__ float2 group_sum(float2 v, Group& g) {
  if constexpr (G == kPacked) return make_float2(packed_sum(v.x, g), packed_sum(v.y, g));
#pragma unroll
  for (int o = width_of(G) / 2; o > 0; o >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if constexpr (warps_of(G)) v = across_warps(v, g);
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v, Group& g) {
  if constexpr (G == kPacked) return packed_sum(v, g);
#pragma unroll
  for (int o = width_of(G) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (warps_of(G)) v = across_warps(make_float2(v, 0.f), g).x;
  return v;
}

template <int G, Layout L>
__device__ __forceinline__ Group make_group(const Params& p, float2 (*smem)[2 * kMaxWarps]) {
  constexpr int W = width_of(G);
  Group g;
  if constexpr (G == kPacked) {
    static_assert(L == kRun, "a part is one run");
    const int per = 32 / p.lanes, at = (int)threadIdx.x & 31, k = at / p.lanes;
    g.lanes = p.lanes;
    g.slots = (int)blockDim.x / 32 * per;
    // the lanes left over: a group behind the last one, without channels (its
    // sums in `red` stay in there: fewer than 8 lanes a warp are left of it)
    g.slot = k < per ? (int)threadIdx.x / 32 * per + k : g.slots;
    g.lane = g.l = at - k * p.lanes;
    g.first = (int)threadIdx.x - g.l;
    g.base = k < per ? 0 : p.C;
    g.c0 = k < per ? kE * g.l : p.C;
    g.c1 = g.c0 + 4;
    g.act = g.c0 < p.C;
    g.buf = nullptr;
    g.turn = 0;
    return g;
  }
  g.lanes = G > 0 ? W : p.lanes;
  g.slots = (int)blockDim.x / g.lanes;
  g.slot = (int)threadIdx.x / g.lanes;
  g.lane = (int)threadIdx.x - g.slot * g.lanes;
  g.l = g.lane % W;
  g.first = (int)threadIdx.x - g.l;
  g.base = (g.lane - g.l) * (kE * parts_of(G));
  g.c0 = g.base + (L == kSplit ? 4 : kE) * g.l;
  g.c1 = g.c0 + (L == kSplit ? 4 * W : 4);
  g.act = L == kSingle || g.c0 < p.C;
  g.buf = G > 0 ? nullptr : smem[g.slot];
  g.turn = 0;
  return g;
}

// v - mean, absent channels kept at zero (a thread without any is left out of
// the sums by Group::act).
template <Layout L, int G, int Q>
__device__ __forceinline__ void centre(Vec<Q>& v, float mean, const Group& g, int C) {
  const float2 m = both(-mean);
#pragma unroll
  for (int k = 0; k < v.P; ++k) v.p[k] = add2(v.p[k], m);
  if constexpr (L == kSingle) {
#pragma unroll
    for (int e = 0; e < v.E; ++e)
      if (channel<L, G>(g, e) >= C) v[e] = 0.f;
  } else if constexpr (L == kSplit || Q > 1) {
    if (C < g.lanes * v.E) {
#pragma unroll
      for (int h = 1; h < 2 * Q; ++h)
        if (run<G>(g, h) >= C) v.p[2 * h] = v.p[2 * h + 1] = both(0.f);
    }
  }
}
template <int Q>
__device__ __forceinline__ void times(Vec<Q>& v, float r) {
#pragma unroll
  for (int k = 0; k < v.P; ++k) v.p[k] = mul2(v.p[k], both(r));
}

// v becomes (v - mean) * rstd (rms: v * rstd); returns rstd.  Two passes over
// registers, the deviations squared after the mean is removed.
template <int G, Layout L, int Q>
__device__ __forceinline__ float standardise(Vec<Q>& v, Group& g, const Params& p) {
  if (!p.rms) {
    const float s = sum(v);
    centre<L, G>(v, group_sum<G>(g.act ? s : 0.f, g) * p.inv_c, g, p.C);
  }
  const float s = dot(v, v);
  const float r = rsqrtf(fmaf(group_sum<G>(g.act ? s : 0.f, g), p.inv_c, p.eps));
  times(v, r);
  return r;
}
// Two rows at once, their sums side by side.
template <int G, Layout L, int Q>
__device__ __forceinline__ float2 standardise(Vec<Q>& a, Vec<Q>& b, Group& g, const Params& p) {
  if (!p.rms) {
    const float2 s = make_float2(sum(a), sum(b));
    const float2 m = group_sum<G>(g.act ? s : both(0.f), g);
    centre<L, G>(a, m.x * p.inv_c, g, p.C);
    centre<L, G>(b, m.y * p.inv_c, g, p.C);
  }
  const float2 s = make_float2(dot(a, a), dot(b, b));
  const float2 t = group_sum<G>(g.act ? s : both(0.f), g);
  const float2 r = make_float2(rsqrtf(fmaf(t.x, p.inv_c, p.eps)), rsqrtf(fmaf(t.y, p.inv_c, p.eps)));
  times(a, r.x);
  times(b, r.y);
  return r;
}

// 1 / (1 + 2^(-v log2 e)): relative error of a few 2^-23 beside |v| 2^-24 of
// the exponent; far below zero the quotient underflows to 0 (v < -87).
template <int Q>
__device__ __forceinline__ void sigmoid(Vec<Q>& v) {
#pragma unroll
  for (int k = 0; k < v.P; ++k) {
    float2 t = mul2(v.p[k], both(-1.4426950408889634f));
    t = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v.p[k].x) : "f"(t.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v.p[k].y) : "f"(t.y));
  }
}
// The sigmoid, and in `away` its distance from 1 as t / (1 + t), t = e^(-v): the
// difference 1 - q would have lost 1e-4 of itself at v = 8 and all at v = 17.
// (Where t overflows or q underflows, the distance is 0 beside q = 0: only their
// product is used.)
template <int Q>
__device__ __forceinline__ void sigmoid(Vec<Q>& v, Vec<Q>& away) {
#pragma unroll
  for (int k = 0; k < v.P; ++k) {
    const float2 e = mul2(v.p[k], both(-1.4426950408889634f));
    const float2 t = make_float2(ex2(e.x), ex2(e.y)), s = add2(t, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v.p[k].x) : "f"(s.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v.p[k].y) : "f"(s.y));
    away.p[k] = mul2(make_float2(fminf(t.x, FLT_MAX), fminf(t.y, FLT_MAX)), v.p[k]);
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename TS, typename TI, int G, bool POST, bool HELD>
struct FwdRing {
  static constexpr int TAKEN = POST ? (HELD ? 1 : 2) : 0;  // of the block's operands
  static constexpr int UNITS = units<TS>() + TAKEN * units<TI>();
  // (UNITS is 1 to 6; three CTAs per SM)
  static constexpr int STAGES = 12 / UNITS > 4 ? 4 : 12 / UNITS;
  __host__ __device__ static constexpr uint32_t stage(uint32_t threads) {
    return ring_bytes<TS, G>(threads) + TAKEN * ring_bytes<TI, G>(threads);
  }
  static constexpr size_t bytes(int threads) { return (size_t)STAGES * stage(threads); }
};

// HELD: a gate row is shared by many consecutive rows; its sigmoid is taken
// when it changes and kept (N = 768, a gate row per 768 rows: 104 us with the
// gate read for every row).
template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE, bool DENSE, bool HELD>
__global__ void __launch_bounds__(threads_of(G), G == kPlain ? 1 : G == kTwice ? 4 : G == kWarpsTwice ? 2 : 3)
    k_block_norm_fwd(const __grid_constant__ Params p) {
  using Ring = FwdRing<TS, TI, G, POST, HELD>;
  extern __shared__ __align__(16) char smem[];
  __shared__ float2 sums[warps_of(G) ? 4 : 1][2 * kMaxWarps];
  wait_for_earlier_work();
  let_next_start();
  constexpr Layout L = layout_of<TS, VEC>();
  using V = Vec<parts_of(G)>;
  constexpr bool CROSS = L == kSplit && sizeof(TI) == 2;  // a warp's threads read each other's copies
  Group g = make_group<G, L>(p, sums);
  const int C = p.C;
  const bool gated = POST && p.gate.p != nullptr;
  const bool shared_gate = p.share > 1;

  constexpr bool CHUNK = !VEC && DENSE;
  const uint32_t chunk_s = chunk_size(g.slots * C, sizeof(TS)), chunk_i = chunk_size(g.slots * C, sizeof(TI));
  const uint32_t stage_bytes = CHUNK ? chunk_s + 2 * chunk_i : Ring::stage(blockDim.x);
  const uint32_t ring_s = smem_u32(smem);
  auto gate_row = [&](uint32_t row, const At<DENSE>& r) {
    return shared_gate ? row_ptr(p.gate, row_pos(p.gate_of, div_by(row, p.by_share)), p.gate_of)
                       : r.block(p, p.gate);
  };
  // this CTA's rows: `turns` of every group, one behind the other
  const uint32_t base = blockIdx.x * g.slots * p.turns;
  const uint32_t last = min(p.rows, base + g.slots * p.turns);
  auto fetch = [&](uint32_t stage, uint32_t row) {
    const bool live = row < last;
    const uint32_t at = live ? row : 0u;
    const At<DENSE> r(p, at);
    uint32_t slot = ring_s + stage * stage_bytes;
    ring_put<TS, L, G>(slot, r.stream(p, p.x), g, C, live);
    if (POST) {
      slot += ring_bytes<TS, G>(blockDim.x);
      ring_put<TI, L, G>(slot, r.block(p, p.u), g, C, live);
      if (!HELD && gated)
        ring_put<TI, L, G>(slot + ring_bytes<TI, G>(blockDim.x), gate_row(at, r), g, C, live);
    }
  };

  auto fetch_chunk = [&](uint32_t stage, uint32_t first) {
    if (first >= last) return;
    const uint32_t n = min(last - first, (uint32_t)g.slots) * C;
    const At<DENSE> r(p, first);
    const uint32_t to = ring_s + stage * stage_bytes;
    const uint32_t ss = (first * p.stride_s) & 15, si = (first * p.stride_i) & 15;
    chunk_put(to, r.stream(p, p.x), n * sizeof(TS), ss);
    if (POST) {
      chunk_put(to + chunk_s, r.block(p, p.u), n * sizeof(TI), si);
      if (gated && !shared_gate) chunk_put(to + chunk_s + chunk_i, r.block(p, p.gate), n * sizeof(TI), si);
    }
  };

  // Every thread of a warp (or of a row's warps) takes part in the sums, so
  // all groups of a CTA make the same number of turns.
  const uint32_t step = g.slots;
  uint32_t turns = (last - base + step - 1) / step;
  uint32_t row = base + g.slot, stage = 0;
  if constexpr (ring_of(G, VEC)) {
#pragma unroll
    for (int s = 0; s < Ring::STAGES - 1; ++s) {
      fetch(s, row + s * step);
      copies_close();
    }
  } else if constexpr (CHUNK) {
    fetch_chunk(0, base);
    copies_close();
  }
  // scale folded into the post-norm's parameters
  V g1, b1, g2, b2;
  if (POST) {
    const V s = param<L, G>(p.scale, 1.f, g, C, p.wide_params);
    g1 = param<L, G>(p.gamma_post, 1.f, g, C, p.wide_params);
    b1 = param<L, G>(p.beta_post, 0.f, g, C, p.wide_params);
#pragma unroll
    for (int k = 0; k < V::P; ++k) {
      g1.p[k] = mul2(g1.p[k], s.p[k]);
      b1.p[k] = mul2(b1.p[k], s.p[k]);
    }
  }
  if (PRE) {
    g2 = param<L, G>(p.gamma_pre, 1.f, g, C, p.wide_params);
    b2 = param<L, G>(p.beta_pre, 0.f, g, C, p.wide_params);
  }

  V held{};
  uint32_t holds = ~0u;  // the gate row that `held` is of
  for (; turns > 0; --turns, row += step) {
    const bool live = row < last;
    const At<DENSE> r(p, live ? row : 0);
    V x, u, q;
    if constexpr (HELD) {
      const uint32_t now = div_by(live ? row : last - 1, p.by_share);
      if (now != holds) {
        holds = now;
        held = load<TI, L, G>(row_ptr(p.gate, row_pos(p.gate_of, now), p.gate_of), g, C);
        sigmoid(held);
      }
    }
    if constexpr (ring_of(G, VEC)) {
      const uint32_t ahead = stage == 0 ? Ring::STAGES - 1 : stage - 1;
      if (CROSS) __syncwarp();  // the warp has read that stage
      fetch(ahead, row + (Ring::STAGES - 1) * step);
      copies_close();
      copies_wait<Ring::STAGES - 1>();
      if (CROSS) __syncwarp();  // what the warp's other threads copied
      const char* slot = smem + stage * stage_bytes;
      x = ring_get<TS, L, G>(slot, g);
      if (POST) {
        slot += ring_bytes<TS, G>(blockDim.x);
        u = ring_get<TI, L, G>(slot, g);
        if (!HELD && gated) q = ring_get<TI, L, G>(slot + ring_bytes<TI, G>(blockDim.x), g);
      }
      stage = stage + 1 == Ring::STAGES ? 0 : stage + 1;
    } else if constexpr (CHUNK) {
      copies_wait<0>();
      __syncthreads();  // the turn's rows are here, and the other stage has been read
      fetch_chunk(stage ^ 1, row - g.slot + step);
      copies_close();
      const char* from = smem + stage * stage_bytes;
      stage ^= 1;
      x = u = q = V{};
      if (live) {
        const uint32_t first = row - g.slot;
        x = load<TS, L, G>(from + ((first * p.stride_s) & 15) + g.slot * C * sizeof(TS), g, C);
        if (POST) {
          from += chunk_s + ((first * p.stride_i) & 15) + g.slot * C * sizeof(TI);
          u = load<TI, L, G>(from, g, C);
          if (gated) q = load<TI, L, G>(shared_gate ? gate_row(row, r) : from + chunk_i, g, C);
        }
      }
    } else {
      x = u = q = V{};
      if (live && g.act) {
        x = load<TS, L, G>(r.stream(p, p.x), g, C);
        if (POST) {
          u = load<TI, L, G>(r.block(p, p.u), g, C);
          if (gated) q = load<TI, L, G>(gate_row(row, r), g, C);
        }
      }
    }
    if (POST) {
      standardise<G, L>(u, g, p);
      if (HELD || gated) {
        if constexpr (HELD) q = held;
        else sigmoid(q);
#pragma unroll
        for (int k = 0; k < V::P; ++k) x.p[k] = fma2(fma2(u.p[k], g1.p[k], b1.p[k]), q.p[k], x.p[k]);
      } else {
#pragma unroll
        for (int k = 0; k < V::P; ++k) x.p[k] = add2(x.p[k], fma2(u.p[k], g1.p[k], b1.p[k]));
      }
      store<TS, L, G>(live, r.stream(p, p.x1), g, C, x);
    }
    if (PRE) {
      standardise<G, L>(x, g, p);
#pragma unroll
      for (int k = 0; k < V::P; ++k) x.p[k] = fma2(x.p[k], g2.p[k], b2.p[k]);
      store<TI, L, G>(live, r.block(p, p.y), g, C, x);
    }
  }
  if constexpr (ring_of(G, VEC) || CHUNK) copies_wait<0>();
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// The rows that a group works on, turn by turn: every `hop`-th row of one
// stretch, or (gate rows shared) of the stretches of its items.  All groups of
// a CTA make the same number of turns; a group out of rows has row >= end.
template <bool GROUPED>
struct Walk {
  uint32_t row, end, hop, left;  // left: turns left in this stretch
  uint32_t item, gate_row;

  __device__ __forceinline__ void open(const Params& p, const Group& g) {
    if constexpr (GROUPED) {
      left = 0;
      if ((p.by_cta ? item : item - g.slot) >= p.items) return;
      const bool mine = item < p.items;
      gate_row = mine ? item / p.segs : 0;
      const uint32_t seg = mine ? item - gate_row * p.segs : 0;
      const uint32_t top = gate_row * p.share;
      row = top + seg * p.seg_rows;
      end = mine ? min(top + p.share, row + p.seg_rows) : row;
      left = p.by_cta ? (end - row + g.slots - 1) / g.slots : p.seg_rows;
      if (p.by_cta) row += g.slot;
    }
  }
  __device__ __forceinline__ void start(const Params& p, const Group& g) {
    if constexpr (GROUPED) {
      hop = p.by_cta ? (uint32_t)g.slots : 1u;
      item = p.by_cta ? blockIdx.x : blockIdx.x * g.slots + g.slot;
      open(p, g);
    } else {
      hop = gridDim.x * g.slots;
      const uint32_t base = blockIdx.x * g.slots;
      row = base + g.slot;
      end = p.rows;
      left = base < p.rows ? (p.rows - base + hop - 1) / hop : 0;
      item = gate_row = 0;
    }
  }
  // To the next turn; true where a stretch ended.
  __device__ __forceinline__ bool advance(const Params& p, const Group& g) {
    row += hop;
    if (--left > 0) return false;
    if constexpr (GROUPED) {
      item += gridDim.x * (p.by_cta ? 1u : (uint32_t)g.slots);
      open(p, g);
    }
    return true;
  }
};

template <typename TS, typename TI, int G, bool POST, bool PRE, bool GROUPED>
struct BwdRing {
  static constexpr int UNITS = units<TS>() * (PRE ? 2 : 1) + (PRE ? units<TI>() : 0) +
                               (POST ? units<TI>() * (GROUPED ? 1 : 2) : 0);
  // One row ahead is enough: with more the rows in flight lie further apart
  // (N = 768, bf16, warps in step: 206 us with 4 stages, 196 with 3, 184 with 2).
  static constexpr int STAGES = 2;
  __host__ __device__ static constexpr uint32_t stage(uint32_t threads) {
    return ring_bytes<TS, G>(threads) * (PRE ? 2 : 1) + (PRE ? ring_bytes<TI, G>(threads) : 0) +
           (POST ? ring_bytes<TI, G>(threads) * (GROUPED ? 1 : 2) : 0);
  }
  static constexpr size_t bytes(int threads) { return (size_t)STAGES * stage(threads); }
};

// Shared memory of the backward: a row of sums per group, three parameter
// vectors by thread of a group, and the ring or the chunks.
constexpr size_t bwd_sums_bytes(int threads, int parts) { return (size_t)threads * kE * 4 * parts; }
constexpr size_t bwd_params_bytes(int lanes, int parts) { return (size_t)lanes * kE * 4 * 3 * parts; }

// CTAs per SM that the registers are cut for.  Two parts per lane need up to
// 255 registers: 8 warps without spills (147,456 rows of 512 bf16 channels:
// 185 us) against 12 with some (208 us); with fp32 rows the 12 are faster
// (98,304 rows of 384 channels: 195 us against 214).
constexpr int resident_bwd(int G, bool fp32) {
  return G == kPlain || G == kWarpsTwice ? 1 : G == kTwice && fp32 ? 3 : 2;
}

// GROUPED: gate rows shared by consecutive rows, whose gradients are summed.
template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE, bool GROUPED,
          bool DENSE>
__global__ void __launch_bounds__(threads_of(G), resident_bwd(G, sizeof(TI) == 4 && VEC && !GROUPED))
    k_block_norm_bwd(const __grid_constant__ Params p) {
  using Ring = BwdRing<TS, TI, G, POST, PRE, GROUPED>;
  extern __shared__ __align__(16) char smem[];
  __shared__ float2 sums[warps_of(G) ? 4 : 1][2 * kMaxWarps];
  wait_for_earlier_work();
  constexpr Layout L = layout_of<TS, VEC>();
  using V = Vec<parts_of(G)>;
  constexpr bool CROSS = L == kSplit && sizeof(TI) == 2;  // a warp's threads read each other's copies
  Group g = make_group<G, L>(p, sums);
  const int C = p.C;
  const bool gated = POST && (GROUPED || p.gate.p != nullptr);
  const bool with_dx1 = p.dx1.p != nullptr;

  constexpr bool RING = ring_of(G, VEC), CHUNK = !VEC && DENSE;
  constexpr bool STEP = RING && (!GROUPED || sizeof(TS) == 4) && G > 0 && G <= 32 && sizeof(TI) == 2;
  const bool in_step = STEP && (!GROUPED || p.in_step);
  float* const red = reinterpret_cast<float*>(smem);  // [slots][lanes * 8]
  // a thread's own 1 - q of a shared gate row, in the sums' place between them
  // (in registers it pushes others out)
  float* const kept = red + threadIdx.x;
  float4* const kept4 = reinterpret_cast<float4*>(smem) + threadIdx.x;
  // parameters: [vector][run][lane] float4, read back without bank conflicts
  float4* const prm = reinterpret_cast<float4*>(smem + bwd_sums_bytes(blockDim.x, parts_of(G)));
  char* const ring = reinterpret_cast<char*>(prm) + bwd_params_bytes(g.lanes, parts_of(G));
  // scale * gamma_post, scale * beta_post, gamma_pre
  auto read = [&](int k) {
    if (k == 2) return param<L, G>(p.gamma_pre, 1.f, g, C, p.wide_params);
    V v = param<L, G>(k == 0 ? p.gamma_post : p.beta_post, k == 0 ? 1.f : 0.f, g, C, p.wide_params);
    const V s = param<L, G>(p.scale, 1.f, g, C, p.wide_params);
#pragma unroll
    for (int j = 0; j < V::P; ++j) v.p[j] = mul2(v.p[j], s.p[j]);
    return v;
  };
  if (g.slot == 0) {
#pragma unroll
    for (int k = POST ? 0 : 2; k < (PRE ? 3 : 2); ++k) {
      const V v = read(k);
#pragma unroll
      for (int h = 0; h < V::P / 2; ++h)
        prm[(k * (V::P / 2) + h) * g.lanes + g.lane] =
            make_float4(v.p[2 * h].x, v.p[2 * h].y, v.p[2 * h + 1].x, v.p[2 * h + 1].y);
    }
  }
  __syncthreads();
  auto get = [&](int k) {
    V v;
#pragma unroll
    for (int h = 0; h < V::P / 2; ++h) put_run(v, h, prm[(k * (V::P / 2) + h) * g.lanes + g.lane]);
    return v;
  };

  const V zero{};
  V acc[4] = {zero, zero, zero, zero};  // sums of D q k, D q, dy h, dy
  V q, dg = zero;  // sigmoid(gate) and the gate's gradient
#pragma unroll
  for (int k = 0; k < V::P; ++k) q.p[k] = both(1.f);

  const uint32_t chunk_s = chunk_size(g.slots * C, sizeof(TS)), chunk_i = chunk_size(g.slots * C, sizeof(TI));
  const uint32_t stage_bytes = CHUNK ? 2 * chunk_s + 3 * chunk_i : Ring::stage(blockDim.x);
  const uint32_t ring_s = smem_u32(ring);
  // ring order: dx1, (x1, dy), (u, gate)
  auto fetch = [&](uint32_t stage, uint32_t row, bool live) {
    const At<DENSE> r(p, live ? row : 0u);
    uint32_t slot = ring_s + stage * stage_bytes;
    if (with_dx1) ring_put<TS, L, G>(slot, r.stream(p, p.dx1), g, C, live);
    slot += ring_bytes<TS, G>(blockDim.x);
    if (PRE) {
      ring_put<TS, L, G>(slot, r.stream(p, p.x), g, C, live);
      slot += ring_bytes<TS, G>(blockDim.x);
      ring_put<TI, L, G>(slot, r.block(p, p.dy), g, C, live);
      slot += ring_bytes<TI, G>(blockDim.x);
    }
    if (POST) {
      ring_put<TI, L, G>(slot, r.block(p, p.u), g, C, live);
      slot += ring_bytes<TI, G>(blockDim.x);
      if (!GROUPED && gated) ring_put<TI, L, G>(slot, r.block(p, p.gate), g, C, live);
    }
  };

  // the rows of the CTA's turn at `w` (a group's row is g.slot rows behind the first)
  auto fetch_chunk = [&](uint32_t stage, const Walk<GROUPED>& w) {
    const uint32_t first = w.row - g.slot;
    if (w.left == 0 || first >= w.end) return;
    const uint32_t n = min(w.end - first, (uint32_t)g.slots) * C;
    const At<DENSE> r(p, first);
    const uint32_t to = ring_s + stage * stage_bytes;
    const uint32_t ss = (first * p.stride_s) & 15, si = (first * p.stride_i) & 15;
    if (with_dx1) chunk_put(to, r.stream(p, p.dx1), n * sizeof(TS), ss);
    if (PRE) {
      chunk_put(to + chunk_s, r.stream(p, p.x), n * sizeof(TS), ss);
      chunk_put(to + 2 * chunk_s, r.block(p, p.dy), n * sizeof(TI), si);
    }
    if (POST) {
      chunk_put(to + 2 * chunk_s + chunk_i, r.block(p, p.u), n * sizeof(TI), si);
      if (!GROUPED && gated) chunk_put(to + 2 * chunk_s + 2 * chunk_i, r.block(p, p.gate), n * sizeof(TI), si);
    }
  };

  Walk<GROUPED> at, ahead;
  at.start(p, g);
  if constexpr (RING) {
    ahead = at;
#pragma unroll
    for (int s = 0; s < Ring::STAGES - 1; ++s) {
      if (ahead.left > 0) {
        fetch(s, ahead.row, ahead.row < ahead.end);
        ahead.advance(p, g);
      }
      copies_close();
    }
  } else if constexpr (CHUNK) {
    ahead = at;
    fetch_chunk(0, ahead);
    copies_close();
  }
  uint32_t stage = 0;
  bool fresh = true;  // a stretch begins
  while (at.left > 0) {
    const uint32_t row = at.row;
    const bool live = row < at.end;  // a group without a row works on zeros
    const At<DENSE> r(p, live ? row : 0);
    if constexpr (GROUPED) {
      if (fresh) {
        const RowPos rg = row_pos(p.gate_of, at.gate_row);
        q = g.act ? load<TI, L, G>(row_ptr(p.gate, rg, p.gate_of), g, C) : zero;
        V away;
        sigmoid(q, away);
        if constexpr (VEC) {
#pragma unroll
          for (int h = 0; h < V::P / 2; ++h)
            kept4[h * blockDim.x] =
                make_float4(away.p[2 * h].x, away.p[2 * h].y, away.p[2 * h + 1].x, away.p[2 * h + 1].y);
        } else {
#pragma unroll
          for (int e = 0; e < V::E; ++e) kept[e * blockDim.x] = away[e];
        }
        dg = zero;
      }
    }
    V D = zero, h, dy, u, gt;
    if constexpr (RING) {
      const uint32_t to = stage == 0 ? Ring::STAGES - 1 : stage - 1;
      // The CTA's warps stay in step: left to themselves they drift apart and the
      // rows in flight with them (N = 768, bf16: 221 us so, 184 in step).  Not
      // where a row takes a warp of its own or several, nor for fp32 rows, where
      // it costs more than it gives; with shared gate rows it may give with an
      // fp32 stream, see launch_bwd.
      if (in_step) __syncthreads();
      if (CROSS) __syncwarp();  // the warp has read that stage
      if (ahead.left > 0) {
        fetch(to, ahead.row, ahead.row < ahead.end);
        ahead.advance(p, g);
      }
      copies_close();
      copies_wait<Ring::STAGES - 1>();
      if (CROSS) __syncwarp();  // what the warp's other threads copied
      const char* slot = ring + stage * stage_bytes;
      if (with_dx1) D = ring_get<TS, L, G>(slot, g);
      slot += ring_bytes<TS, G>(blockDim.x);
      if (PRE) {
        h = ring_get<TS, L, G>(slot, g);
        slot += ring_bytes<TS, G>(blockDim.x);
        dy = ring_get<TI, L, G>(slot, g);
        slot += ring_bytes<TI, G>(blockDim.x);
      }
      if (POST) {
        u = ring_get<TI, L, G>(slot, g);
        if (!GROUPED && gated) gt = ring_get<TI, L, G>(slot + ring_bytes<TI, G>(blockDim.x), g);
      }
      stage = stage + 1 == Ring::STAGES ? 0 : stage + 1;
    } else if constexpr (CHUNK) {
      copies_wait<0>();
      __syncthreads();  // the turn's rows are here, and the other stage has been read
      ahead.advance(p, g);
      fetch_chunk(stage ^ 1, ahead);
      copies_close();
      const uint32_t first = row - g.slot;
      const char* from = ring + stage * stage_bytes;
      stage ^= 1;
      h = dy = u = gt = zero;
      if (live) {
        const char* at_s = from + ((first * p.stride_s) & 15) + g.slot * C * sizeof(TS);
        if (with_dx1) D = load<TS, L, G>(at_s, g, C);
        if (PRE) h = load<TS, L, G>(at_s + chunk_s, g, C);
        from += 2 * chunk_s + ((first * p.stride_i) & 15) + g.slot * C * sizeof(TI);
        if (PRE) dy = load<TI, L, G>(from, g, C);
        if (POST) {
          u = load<TI, L, G>(from + chunk_i, g, C);
          if (!GROUPED && gated) gt = load<TI, L, G>(from + 2 * chunk_i, g, C);
        }
      }
    } else {
      auto stream = [&](const Operand& o) {
        return live && g.act ? load<TS, L, G>(r.stream(p, o), g, C) : zero;
      };
      auto block = [&](const Operand& o) {
        return live && g.act ? load<TI, L, G>(r.block(p, o), g, C) : zero;
      };
      if (with_dx1) D = stream(p.dx1);
      if (PRE) {
        h = stream(p.x);
        dy = block(p.dy);
      }
      if (POST) {
        u = block(p.u);
        if (!GROUPED && gated) gt = block(p.gate);
      }
    }

    float2 rstd = both(0.f);  // of x1 and of u
    if (PRE && POST) rstd = standardise<G, L>(h, u, g, p);
    else if (PRE) rstd.x = standardise<G, L>(h, g, p);
    else rstd.y = standardise<G, L>(u, g, p);
    if (PRE) {
      const V g2 = get(2);
#pragma unroll
      for (int k = 0; k < V::P; ++k) {
        acc[2].p[k] = fma2(dy.p[k], h.p[k], acc[2].p[k]);
        acc[3].p[k] = add2(acc[3].p[k], dy.p[k]);
        dy.p[k] = mul2(dy.p[k], g2.p[k]);
      }
      float2 s = make_float2(sum(dy), dot(dy, h));
      s = group_sum<G>(g.act ? s : both(0.f), g);
      const float2 m0 = both(p.rms ? 0.f : -s.x * p.inv_c), m1 = both(-s.y * p.inv_c), rs = both(rstd.x);
#pragma unroll
      for (int k = 0; k < V::P; ++k)
        D.p[k] = fma2(rs, fma2(m1, h.p[k], add2(dy.p[k], m0)), D.p[k]);
      store<TS, L, G>(live, r.stream(p, p.dx), g, C, D);
    }
    if (POST) {
      const V g1 = get(0), b1 = get(1);
      if (!GROUPED && gated) {
        V away;
        q = gt;
        sigmoid(q, away);
#pragma unroll
        for (int k = 0; k < V::P; ++k) {
          D.p[k] = mul2(D.p[k], q.p[k]);
          const float2 w = fma2(u.p[k], g1.p[k], b1.p[k]);  // (with the scale)
          dg.p[k] = mul2(mul2(D.p[k], w), away.p[k]);
        }
      }
      V b;
#pragma unroll
      for (int k = 0; k < V::P; ++k) {
        const float2 dq = GROUPED ? mul2(D.p[k], q.p[k]) : D.p[k];
        acc[0].p[k] = fma2(dq, u.p[k], acc[0].p[k]);
        acc[1].p[k] = add2(acc[1].p[k], dq);
        // (1 - q) is applied once, at the end
        if (GROUPED) dg.p[k] = fma2(dq, fma2(u.p[k], g1.p[k], b1.p[k]), dg.p[k]);
        b.p[k] = mul2(dq, g1.p[k]);
      }
      float2 s = make_float2(sum(b), dot(b, u));
      s = group_sum<G>(g.act ? s : both(0.f), g);
      const float2 m0 = both(p.rms ? 0.f : -s.x * p.inv_c), m1 = both(-s.y * p.inv_c), rs = both(rstd.y);
#pragma unroll
      for (int k = 0; k < V::P; ++k) b.p[k] = mul2(rs, fma2(m1, u.p[k], add2(b.p[k], m0)));
      store<TI, L, G>(live, r.block(p, p.du), g, C, b);
      if (!GROUPED && gated) store<TI, L, G>(live, r.block(p, p.dgate), g, C, dg);
    }

    const Walk<GROUPED> was = at;
    fresh = at.advance(p, g);
    if constexpr (GROUPED) {
      if (fresh) {
        if constexpr (VEC) {
#pragma unroll
          for (int h = 0; h < V::P / 2; ++h) {
            const float4 away = kept4[h * blockDim.x];
            dg.p[2 * h] = mul2(dg.p[2 * h], make_float2(away.x, away.y));
            dg.p[2 * h + 1] = mul2(dg.p[2 * h + 1], make_float2(away.z, away.w));
          }
        } else {
#pragma unroll
          for (int e = 0; e < V::E; ++e) dg[e] *= kept[e * blockDim.x];
        }
        const RowPos rg = row_pos(p.gate_of, was.gate_row);
        char* const whole = row_ptr(p.dgate, rg, p.gate_of);
        float* const part = p.gate_part + (size_t)was.item * C;  // (where segs > 1)
        if (p.by_cta && g.slots > 1) {
          // a thread per channel adds the groups' sums (a group's threads,
          // eight channels each: 589,824 bf16 rows of 32 74 us, 62 so)
          const int width = g.lanes * V::E;
          __syncthreads();
#pragma unroll
          for (int e = 0; e < V::E; ++e) red[g.slot * width + channel<L, G>(g, e)] = dg[e];
          __syncthreads();
          for (int c = threadIdx.x; c < C; c += blockDim.x) {
            float s = 0.f;
            for (int i = 0; i < g.slots; ++i) s += red[i * width + c];
            if (p.segs == 1) reinterpret_cast<TI*>(whole)[c] = static_cast<TI>(s);
            else part[c] = s;
          }
          __syncthreads();  // `kept` takes their place
        } else {
          const bool writes = p.by_cta || was.item < p.items;
          if (p.segs == 1) store<TI, L, G>(writes, whole, g, C, dg);
          else store<float, L, G>(writes, reinterpret_cast<char*>(part), g, C, dg);
        }
      }
    }
  }

  let_next_start();
  // the CTA's sums, group by group in order
  const int width = g.lanes * V::E;
#pragma unroll
  for (int k = POST ? 0 : 2; k < (PRE ? 4 : 2); ++k) {
    if (!p.wanted[k >> 1]) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V::E; ++e) red[g.slot * width + channel<L, G>(g, e)] = acc[k][e];
    __syncthreads();
    float* dst = p.part + ((size_t)blockIdx.x * kSums + k) * C;
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
// Resident CTAs of a kernel per SM times the SMs, looked up once per device
// and number of lanes that share a row: a CTA's threads and shared memory
// follow from it.  (From the threads alone the latter does not: fp32 rows of
// 1001 and of 2047 channels both have 256, two and one CTAs per SM.)  `most` is
// the shared memory of the kernel's largest CTA.
template <typename K>
cudaError_t resident_ctas(K kernel, int lanes, int threads, size_t smem, size_t most,
                          std::atomic<int> (&cache)[64][17], int* n) {
  const int key = lanes % 32 ? lanes : lanes / 32;  // (a kernel has either kind)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64) *n = cache[dev][key].load(std::memory_order_relaxed);
  else *n = 0;
  if (*n > 0) return cudaSuccess;
  int sms = 0, per = 0;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *n = std::max(1, sms) * std::max(1, per);
  if (dev >= 0 && dev < 64) cache[dev][key].store(*n, std::memory_order_relaxed);
  return cudaSuccess;
}

// The launch's row space.  Axes along which the gate repeats its rows come
// last, so that a gate row's rows are consecutive; the others are ordered by
// the stride of the first operand given.
struct Axis {
  uint32_t n;
  int64_t s[10];
  bool shared;
};
struct Space {
  Axis ax[3];
  int count;
  uint32_t share;
};
inline Space order_axes(const int (&n)[3], const RowOperand* const* ops, int count, int gate_at) {
  Space sp{};
  for (int d = 0; d < 3; ++d) {
    if (n[d] == 1) continue;
    Axis& a = sp.ax[sp.count++];
    a.n = (uint32_t)n[d];
    for (int i = 0; i < count; ++i) a.s[i] = ops[i]->p ? ops[i]->s[d] : 0;
    a.shared = gate_at >= 0 && a.s[gate_at] == 0;
  }
  int lead = 0;
  while (lead + 1 < count && !ops[lead]->p) ++lead;
  std::stable_sort(sp.ax, sp.ax + sp.count, [lead](const Axis& a, const Axis& b) {
    if (a.shared != b.shared) return !a.shared;
    return a.s[lead] > b.s[lead];
  });
  sp.share = 1;
  for (int d = 0; d < sp.count; ++d)
    if (sp.ax[d].shared) sp.share *= sp.ax[d].n;
  return sp;
}

// Three axes (the innermost last) of the operands in `use`: neighbouring axes
// that all of them walk as one become one.  `own_rows`: without the axes along
// which the gate repeats.
inline Rows join_axes(const Space& sp, const RowOperand* const* ops, Operand* const* dst,
                      const int* esize, int count, const bool* use, bool own_rows) {
  Axis ax[3];
  int m = 0;
  for (int d = 0; d < sp.count; ++d) {
    if (own_rows && sp.ax[d].shared) continue;
    bool join = m > 0;
    for (int i = 0; join && i < count; ++i)
      if (use[i] && ops[i]->p) join = ax[m - 1].s[i] == sp.ax[d].s[i] * (int64_t)sp.ax[d].n;
    if (join) {
      const uint32_t outer = ax[m - 1].n;
      ax[m - 1] = sp.ax[d];
      ax[m - 1].n = outer * sp.ax[d].n;
    } else {
      ax[m++] = sp.ax[d];
    }
  }
  uint32_t n[3];
  for (int d = 0; d < 3; ++d) {  // right-aligned
    const int from = d - (3 - m);
    n[d] = from >= 0 ? ax[from].n : 1u;
    for (int i = 0; i < count; ++i) {
      if (!use[i] || !ops[i]->p) continue;
      int64_t& s = d == 0 ? dst[i]->s0 : d == 1 ? dst[i]->s1 : dst[i]->s2;
      s = from >= 0 ? ax[from].s[i] * esize[i] : 0;
    }
  }
  return Rows{fast_div(n[2]), fast_div(n[1]), n[0] == 1 && n[1] == 1};
}

struct Plan {
  Params p;
  int g;        // lanes of a row's group: 8, 16, 32, or kTwice, kWarps, kWarpsTwice, kPlain
  bool vec, dense, chunk;
  int threads, slots;
};

// Sizes and operands, for both directions: `ops` go to `dst` (parts of pl.p),
// their element sizes in `esize`; the gate and its gradient (`is_gate`) have
// row axes of their own where gate rows are shared.  `is_stream`: operands of
// the residual stream.
inline void make_plan(const BlockNormCall& c, const RowOperand* const* ops, Operand* const* dst,
                      const int* esize, const bool* is_stream, const bool* is_gate, int count,
                      int gate_at, bool backward, Plan& pl) {
  Params& p = pl.p;
  const Space sp = order_axes(c.n, ops, count, c.gate.p ? gate_at : -1);
  p.share = sp.share;
  bool rows[10], gates[10];
  for (int i = 0; i < count; ++i) {
    gates[i] = is_gate[i] && sp.share > 1;
    rows[i] = !gates[i];
  }
  p.rows_of = join_axes(sp, ops, dst, esize, count, rows, false);
  p.gate_of = join_axes(sp, ops, dst, esize, count, gates, true);
  p.by_share = fast_div(sp.share);
  p.rows = (uint32_t)((int64_t)c.n[0] * c.n[1] * c.n[2]);
  pl.vec = c.C % kE == 0;
  for (int i = 0; i < count; ++i) {
    Operand& o = *dst[i];
    o.p = static_cast<char*>(ops[i]->p);
    if (o.p && (reinterpret_cast<uintptr_t>(o.p) % 16 || o.s0 % 16 || o.s1 % 16 || o.s2 % 16)) pl.vec = false;
  }
  int64_t stride[2] = {-1, -1};
  pl.dense = p.rows_of.flat;
  for (int i = 0; i < count; ++i) {
    if (!rows[i] || !dst[i]->p) continue;
    int64_t& st = stride[is_stream[i] ? 0 : 1];
    if (st < 0) st = dst[i]->s2;
    if (dst[i]->s2 != st || st > 0xFFFFFFFFll) pl.dense = false;
  }
  p.stride_s = (uint32_t)std::max<int64_t>(stride[0], 0);
  p.stride_i = (uint32_t)std::max<int64_t>(stride[1], 0);
  p.C = c.C;
  p.rms = c.rms;
  p.eps = c.eps;
  p.inv_c = 1.0f / (float)c.C;
  p.scale = c.scale;
  p.gamma_post = c.gamma_post;
  p.beta_post = c.beta_post;
  p.gamma_pre = c.gamma_pre;
  p.beta_pre = c.beta_pre;
  p.wide_params = true;
  for (const float* v : {c.scale, c.gamma_post, c.beta_post, c.gamma_pre, c.beta_pre})
    if (reinterpret_cast<uintptr_t>(v) % 16) p.wide_params = false;
  const int need = (c.C + kE - 1) / kE;  // threads of a row
  if (need <= 32) {
    // (147,456 bf16 rows of 101, one element per access: a warp per row 88 us
    // forward and 126 backward, 16 lanes 49 and 76)
    pl.g = need <= 8 ? 8 : need <= 16 ? 16 : 32;
    p.lanes = pl.g;
    pl.threads = kThreads;
  } else if (need <= kTwice) {
    pl.g = kTwice;
    p.lanes = 32;
    pl.threads = threads_of(kTwice);
  } else {
    // Two parts per lane need fewer instructions and barriers per channel, but
    // more registers: from 1024 channels on the backward gains (49,152 bf16
    // rows of 2048: 347 -> 307 us) and the bf16 forward (255 -> 239), below
    // both lose (98,304 rows of 768: 270 -> 299, 171 -> 195); the forward with
    // an fp32 stream is faster with one part (24,576 fp32 rows of 2048: 149,
    // 171 with two).
    const bool two = pl.vec && (need > kThreads || (need >= 128 && (backward || esize[0] == 2)));
    pl.g = two ? kWarpsTwice : pl.vec ? kWarps : kPlain;
    const int warps = two ? (need + 63) / 64 : (need + 31) / 32;
    p.lanes = warps * 32;
    pl.threads = p.lanes * std::max(1, (two ? 4 : kThreads / 32) / warps);
  }
  pl.slots = pl.threads / p.lanes;
  // A group of as many lanes as a row has parts, where a warp holds more rows
  // so (bf16 rows, forward and backward: 589,824 of 32 51 -> 33 and 91 -> 57 us,
  // 200,000 of 80 38 -> 33 and 66 -> 58).
  if (pl.vec && esize[0] == 2 && need <= 16 && 32 / need > 32 / p.lanes) {
    pl.g = kPacked;
    p.lanes = need;
    pl.slots = pl.threads / 32 * (32 / need);
  }
  // rows one behind the other
  pl.chunk = !pl.vec && pl.dense;
  for (int i = 0; i < count && pl.chunk; ++i)
    if (rows[i] && dst[i]->p)
      pl.chunk = dst[i]->s2 == (int64_t)c.C * esize[i] && reinterpret_cast<uintptr_t>(dst[i]->p) % 16 == 0;
}

// Sums of the CTAs' partial sums: one block per 32 columns of the post-norm's
// sums, of the pre-norm's, or of one gate row, 32 warps taking every 32nd
// partial sum.
constexpr int kReduceWarps = 32;
template <typename TI>
__global__ void __launch_bounds__(kReduceWarps * 32)
    k_block_norm_reduce(const __grid_constant__ Params p, int ctas, int param_blocks) {
  __shared__ float2 red[kReduceWarps][32];
  wait_for_earlier_work();
  const int per = (p.C + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_param = (int)blockIdx.x < param_blocks;
  const int blk = is_param ? blockIdx.x : blockIdx.x - param_blocks;
  const int what = blk / per, c = (blk - what * per) * 32 + lane;
  if (is_param && !p.wanted[what]) return;
  float2 s = both(0.f);
  if (c < p.C) {
    if (is_param) {
      const float* src = p.part + (size_t)(2 * what) * p.C + c;
#pragma unroll 4
      for (int i = warp; i < ctas; i += kReduceWarps) {
        const float* at = src + (size_t)i * kSums * p.C;
        s = add2(s, make_float2(at[0], at[p.C]));
      }
    } else {
      const float* src = p.gate_part + (size_t)what * p.segs * p.C + c;
#pragma unroll 4
      for (int i = warp; i < (int)p.segs; i += kReduceWarps) s.x += src[(size_t)i * p.C];
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= p.C) return;
#pragma unroll
  for (int i = 1; i < kReduceWarps; ++i) s = add2(s, red[i][lane]);
  if (!is_param) {
    char* row = row_ptr(p.dgate, row_pos(p.gate_of, (uint32_t)what), p.gate_of);
    reinterpret_cast<TI*>(row)[c] = static_cast<TI>(s.x);
  } else if (what == 0) {
    const float sc = p.scale ? p.scale[c] : 1.f;
    if (p.dscale)
      p.dscale[c] = (p.gamma_post ? p.gamma_post[c] : 1.f) * s.x + (p.beta_post ? p.beta_post[c] : 0.f) * s.y;
    if (p.dgamma_post) p.dgamma_post[c] = sc * s.x;
    if (p.dbeta_post) p.dbeta_post[c] = sc * s.y;
  } else {
    if (p.dgamma_pre) p.dgamma_pre[c] = s.x;
    if (p.dbeta_pre) p.dbeta_pre[c] = s.y;
  }
}

// Two stages of chunks: `of_s` operands of the stream and `of_i` of the block,
// at the most channels that a CTA's turn can have.
template <typename TS, typename TI>
constexpr size_t chunk_bytes(int threads, int parts, int of_s, int of_i) {
  return 2 * ((size_t)of_s * chunk_size(threads * kE * parts, sizeof(TS)) +
              (size_t)of_i * chunk_size(threads * kE * parts, sizeof(TI)));
}

template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE, bool DENSE, bool HELD = false>
cudaError_t launch_fwd(Plan pl, cudaStream_t st) {
  static std::atomic<int> cache[64][17];
  auto kern = k_block_norm_fwd<TS, TI, G, VEC, POST, PRE, DENSE, HELD>;
  using Ring = FwdRing<TS, TI, G, POST, HELD>;
  constexpr bool RING = ring_of(G, VEC);
  constexpr bool CHUNK = !VEC && DENSE;
  auto ring = [](int threads) {
    return RING ? Ring::bytes(threads) : CHUNK ? chunk_bytes<TS, TI>(threads, parts_of(G), 1, 2) : 0;
  };
  const size_t smem = ring(pl.threads);
  int ctas = 0;
  cudaError_t e = resident_ctas(kern, pl.p.lanes, pl.threads, smem, ring(threads_of(G)), cache, &ctas);
  if (e != cudaSuccess) return e;
  // The CTAs are many and short (up to 8 turns), so that the rows that are in
  // flight lie close together: CTAs that walk the rows with a stride of the
  // grid drift apart, which costs a fifth of the memory rate (N = 768, bf16:
  // 136 us so, 113 with 8 turns per CTA).
  Params p = pl.p;
  const unsigned need = (p.rows + pl.slots - 1) / pl.slots;
  p.turns = std::max(1u, std::min<unsigned>(8, need / (unsigned)ctas));
  const unsigned per_cta = pl.slots * p.turns;
  return launch_early(kern, (p.rows + per_cta - 1) / per_cta, pl.threads, smem, st, p);
}

template <typename TS, typename TI, int G, bool VEC, bool POST, bool PRE, bool GROUPED, bool DENSE>
cudaError_t launch_bwd(Plan pl, float* ws, cudaStream_t st) {
  static std::atomic<int> cache[64][17];
  auto kern = k_block_norm_bwd<TS, TI, G, VEC, POST, PRE, GROUPED, DENSE>;
  Params& p = pl.p;
  using Ring = BwdRing<TS, TI, G, POST, PRE, GROUPED>;
  constexpr bool RING = ring_of(G, VEC);
  constexpr int Q = parts_of(G);
  constexpr bool CHUNK = !VEC && DENSE;
  const size_t smem = bwd_sums_bytes(pl.threads, Q) + bwd_params_bytes(p.lanes, Q) +
                      (RING ? Ring::bytes(pl.threads) : CHUNK ? chunk_bytes<TS, TI>(pl.threads, Q, 2, 3) : 0);
  constexpr int T = threads_of(G);
  constexpr size_t most = bwd_sums_bytes(T, Q) + bwd_params_bytes(std::max(T, 32), Q) +
                          (RING ? Ring::bytes(T) : CHUNK ? chunk_bytes<TS, TI>(T, Q, 2, 3) : 0);
  static_assert(most <= 227 * 1024 - 2048, "shared memory");
  int ctas = 0;
  cudaError_t e = resident_ctas(kern, p.lanes, pl.threads, smem, most, cache, &ctas);
  if (e != cudaSuccess) return e;
  ctas = std::min(ctas, kNormMaxCtas);
  unsigned need = (p.rows + pl.slots - 1) / pl.slots;
  if (GROUPED) {
    // A gate row's rows are walked by one group where they are fewer than the
    // CTA's groups (spreading them would leave groups idle), else spread over
    // a CTA, in as many items per gate row as give the CTAs the fewest turns:
    // one item each for a few gate rows, several where whole gate rows would
    // leave CTAs without one in the last round.  (An item's end costs about
    // three turns.)
    const uint32_t gates = p.rows / p.share;
    p.by_cta = p.share >= (uint32_t)pl.slots;
    p.segs = 1;
    p.seg_rows = p.share;
    if (p.by_cta) {
      const uint32_t slots = pl.slots, n = ctas;
      const auto up = [](uint64_t a, uint64_t b) { return (a + b - 1) / b; };
      uint64_t least = up(gates, n) * (up(p.share, slots) + 3);
      for (uint32_t rounds = 1; rounds <= 8; ++rounds) {
        const uint64_t segs = std::min<uint64_t>((uint64_t)rounds * n, kNormMaxItems) / gates;
        if (segs < 2) continue;
        const uint64_t turns = up(up(p.share, segs), slots);
        if (rounds * (turns + 3) >= least) continue;
        least = rounds * (turns + 3);
        p.seg_rows = (uint32_t)(turns * slots);
        p.segs = (uint32_t)up(p.share, p.seg_rows);
      }
    }
    // In step where a stretch has many turns and the rows fill their lanes
    // (fp32 stream, us apart and in step: 589,824 rows of 128 with one gate row
    // 227 and 205, with a gate row per 768, 48 turns, 224 and 222; a gate row
    // per 512, 32 turns, 101 and 106, rows of 112 with one per 585 108 and 121;
    // 196,608 rows of 192 with one per 512, lanes three quarters full, 133 and 136).
    p.in_step = p.by_cta && p.seg_rows >= 48u * (uint32_t)pl.slots && p.C > 6 * p.lanes;
    p.items = gates * p.segs;
    need = p.by_cta ? p.items : (p.items + pl.slots - 1) / pl.slots;
  }
  const unsigned grid = std::min<unsigned>(need, (unsigned)ctas);
  p.part = ws;
  p.gate_part = ws + (size_t)kNormMaxCtas * kSums * p.C;
  e = launch_early(kern, grid, pl.threads, smem, st, p);
  if (e != cudaSuccess) return e;
  const int per = (p.C + 31) / 32;
  const int param_blocks = p.wanted[0] || p.wanted[1] ? 2 * per : 0;
  const int gate_blocks = GROUPED && p.segs > 1 ? (int)(p.rows / p.share) * per : 0;
  if (param_blocks + gate_blocks > 0) {
    e = launch_early(k_block_norm_reduce<TI>, param_blocks + gate_blocks, kReduceWarps * 32, 0, st, p, (int)grid,
                     param_blocks);
  }
  return e;
}

template <typename TS, typename TI, bool POST, bool PRE, bool DENSE, bool HELD>
cudaError_t ring_fwd(const Plan& pl, cudaStream_t st) {
  if constexpr (sizeof(TS) == 2)
    if (pl.g == kPacked) return launch_fwd<TS, TI, kPacked, true, POST, PRE, DENSE, HELD>(pl, st);
  switch (pl.g) {
    case 8: return launch_fwd<TS, TI, 8, true, POST, PRE, DENSE, HELD>(pl, st);
    case 16: return launch_fwd<TS, TI, 16, true, POST, PRE, DENSE, HELD>(pl, st);
    case 32: return launch_fwd<TS, TI, 32, true, POST, PRE, DENSE, HELD>(pl, st);
    case kTwice: return launch_fwd<TS, TI, kTwice, true, POST, PRE, DENSE, HELD>(pl, st);
    case kWarps: return launch_fwd<TS, TI, kWarps, true, POST, PRE, DENSE, HELD>(pl, st);
    default: return launch_fwd<TS, TI, kWarpsTwice, true, POST, PRE, DENSE, HELD>(pl, st);
  }
}
template <typename TS, typename TI, bool POST, bool PRE, bool CHUNK>
cudaError_t single_fwd(const Plan& pl, cudaStream_t st) {
  switch (pl.g) {
    case 8: return launch_fwd<TS, TI, 8, false, POST, PRE, CHUNK>(pl, st);
    case 16: return launch_fwd<TS, TI, 16, false, POST, PRE, CHUNK>(pl, st);
    case 32: return launch_fwd<TS, TI, 32, false, POST, PRE, CHUNK>(pl, st);
    case kTwice: return launch_fwd<TS, TI, kTwice, false, POST, PRE, CHUNK>(pl, st);
    default: return launch_fwd<TS, TI, kPlain, false, POST, PRE, CHUNK>(pl, st);
  }
}
template <typename TS, typename TI, bool POST, bool PRE>
cudaError_t dispatch_fwd(const Plan& pl, cudaStream_t st) {
  if (pl.vec) {
    if constexpr (POST) {  // a gate row for at least the rows of a CTA
      if (pl.p.gate.p && pl.p.share >= 8u * (uint32_t)pl.slots)
        return pl.dense ? ring_fwd<TS, TI, POST, PRE, true, true>(pl, st)
                        : ring_fwd<TS, TI, POST, PRE, false, true>(pl, st);
    }
    return pl.dense ? ring_fwd<TS, TI, POST, PRE, true, false>(pl, st)
                    : ring_fwd<TS, TI, POST, PRE, false, false>(pl, st);
  }
  return pl.chunk ? single_fwd<TS, TI, POST, PRE, true>(pl, st) : single_fwd<TS, TI, POST, PRE, false>(pl, st);
}

template <typename TS, typename TI, bool POST, bool PRE, bool GROUPED, bool DENSE>
cudaError_t ring_bwd(const Plan& pl, float* ws, cudaStream_t st) {
  if constexpr (sizeof(TS) == 2)
    if (pl.g == kPacked) return launch_bwd<TS, TI, kPacked, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
  switch (pl.g) {
    case 8: return launch_bwd<TS, TI, 8, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
    case 16: return launch_bwd<TS, TI, 16, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
    case 32: return launch_bwd<TS, TI, 32, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
    case kTwice: return launch_bwd<TS, TI, kTwice, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
    case kWarps: return launch_bwd<TS, TI, kWarps, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
    default: return launch_bwd<TS, TI, kWarpsTwice, true, POST, PRE, GROUPED, DENSE>(pl, ws, st);
  }
}
template <typename TS, typename TI, bool POST, bool PRE, bool GROUPED, bool CHUNK>
cudaError_t single_bwd(const Plan& pl, float* ws, cudaStream_t st) {
  switch (pl.g) {
    case 8: return launch_bwd<TS, TI, 8, false, POST, PRE, GROUPED, CHUNK>(pl, ws, st);
    case 16: return launch_bwd<TS, TI, 16, false, POST, PRE, GROUPED, CHUNK>(pl, ws, st);
    case 32: return launch_bwd<TS, TI, 32, false, POST, PRE, GROUPED, CHUNK>(pl, ws, st);
    case kTwice: return launch_bwd<TS, TI, kTwice, false, POST, PRE, GROUPED, CHUNK>(pl, ws, st);
    default: return launch_bwd<TS, TI, kPlain, false, POST, PRE, GROUPED, CHUNK>(pl, ws, st);
  }
}
template <typename TS, typename TI, bool POST, bool PRE, bool GROUPED>
cudaError_t dispatch_bwd(const Plan& pl, float* ws, cudaStream_t st) {
  if (pl.vec)
    return pl.dense ? ring_bwd<TS, TI, POST, PRE, GROUPED, true>(pl, ws, st)
                    : ring_bwd<TS, TI, POST, PRE, GROUPED, false>(pl, ws, st);
  // (with shared gate rows the rows of a CTA's turn are one piece where a
  // gate row's rows are spread over the CTA, see launch_bwd: 200,000 bf16 rows
  // of 99 with a gate row per 256: 204 us read one by one, 103 so)
  if (pl.chunk && (!GROUPED || pl.p.share >= (uint32_t)pl.slots))
    return single_bwd<TS, TI, POST, PRE, GROUPED, true>(pl, ws, st);
  return single_bwd<TS, TI, POST, PRE, GROUPED, false>(pl, ws, st);
}

template <typename TS, typename TI>
cudaError_t run_fwd(const BlockNormCall& c, cudaStream_t st) {
  constexpr int S = sizeof(TS), I = sizeof(TI);
  Plan pl{};
  Params& p = pl.p;
  const RowOperand* ops[] = {&c.x, &c.u, &c.gate, &c.x1, &c.y};
  Operand* dst[] = {&p.x, &p.u, &p.gate, &p.x1, &p.y};
  const int es[] = {S, I, I, S, I};
  const bool stream[] = {true, false, false, true, false};
  const bool gates[] = {false, false, true, false, false};
  make_plan(c, ops, dst, es, stream, gates, 5, 2, false, pl);
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
  const bool stream[] = {true, true, false, false, false, true, false, false};
  const bool gates[] = {false, false, false, true, false, false, false, true};
  make_plan(c, ops, dst, es, stream, gates, 8, 3, true, pl);
  p.dscale = c.dscale;
  p.dgamma_post = c.dgamma_post;
  p.dbeta_post = c.dbeta_post;
  p.dgamma_pre = c.dgamma_pre;
  p.dbeta_pre = c.dbeta_pre;
  p.wanted[0] = c.dscale || c.dgamma_post || c.dbeta_post;
  p.wanted[1] = c.dgamma_pre || c.dbeta_pre;
  const bool grouped = c.gate.p && p.share > 1;
  if (c.u.p && c.dy.p)
    return grouped ? dispatch_bwd<TS, TI, true, true, true>(pl, c.ws, st)
                   : dispatch_bwd<TS, TI, true, true, false>(pl, c.ws, st);
  if (c.u.p)
    return grouped ? dispatch_bwd<TS, TI, true, false, true>(pl, c.ws, st)
                   : dispatch_bwd<TS, TI, true, false, false>(pl, c.ws, st);
  return dispatch_bwd<TS, TI, false, true, false>(pl, c.ws, st);
}

}  // namespace
}  // namespace norm
}  // namespace evo
