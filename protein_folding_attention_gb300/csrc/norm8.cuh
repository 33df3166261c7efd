// The residual add with dropout, the norm with 8-bit output behind it, and the
// gradients of both:
//
//   x1 = x + keep * u / (1 - p)            y = n(x1) * gamma + beta
//   codes, scales: y in e4m3 with a power of two for each 128 channels
//
//   with h = n(x1), r = 1 / sqrt(var + eps), e = dy * gamma:
//   D  = dx1 + r (e - h mean(e h) - mean(e))     (the last mean: layer norm only)
//   dx = D    du = keep * D / (1 - p)    dgamma = sum dy h    dbeta = sum dy
//
// All of it is bound by memory: each operand is touched once, a row stays in
// registers between its sums and its stores, and the mask is drawn again
// wherever it is needed (philox.cuh).  What the memory rate leaves at bf16 is some
// 30 instructions per element, of which a block of the generator for four
// elements takes 15; so
// - a thread holds T rows at once (their loads in flight together, their sums
//   interleaved), and where rows share a mask these are T rows that do, so that
//   it is drawn once for them;
// - divisions by extents are multiplications, and operands whose rows lie evenly
//   spaced (FLAT) need none;
// - arithmetic goes over pairs of fp32.
// Measured (device time; of the copy rate): forward, 589,824 bf16 rows of 128 98 us
// with a mask shared along i (79 %), 82 without dropout (95 %); 196,608 rows of 384
// 123 with a mask of their own and 87 without (63, 89 %); 262,144 fp32 rows of 128 72
// (90 %).  Backward, 589,824 rows 132 (84 %), 147,456 rows of the ending node's views 41
// (68 %: starting, draining and the second kernel are a third of it), fp32 108 (91 %).
// Rows of odd widths are bound by their single-element accesses: 147,456 bf16 rows
// of 131 106 and 112 us (19, 25 %).
//
// A row lies over LANES threads.  Rows of whole 16-byte units (C % 8 == 0,
// aligned): a thread holds parts of 8 consecutive channels, so 16 neighbouring
// threads hold a group of 128 and its maximum is four shuffles.  Any other
// rows: a warp holds whole groups, each thread every 32nd channel of one, so
// that accesses of single elements are still consecutive across the warp.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "divide.cuh"
#include "launch.cuh"
#include "norm8.h"
#include "philox.cuh"
#include "scale8.cuh"

namespace evo {
namespace norm8 {

struct Params {
  uint32_t rows;
  Divide n1, n2;     // row r = (b * n1 + i) * n2 + j, axes merged where the operands allow it
  Divide I, J;       // the same on the axes as they were given, for the mask
  // Groups of T rows: consecutive ones, or (along_i) T neighbours along axis I
  // with the same j, which share a mask row.
  bool along_i, shared;  // shared: a row's index is not its mask row's
  uint32_t blocks_i;     // ceil(I / T)
  Divide by_blocks_i;
  uint32_t groups;       // of rows
  int C;
  float inv_c, eps;
  bool rms, drop;
  DropMask mask;
  RowOperand x, u, x1, dx1, dy, dx, du;
  uint8_t* codes;
  int64_t codes_s[3];
  uint8_t* scales;
  int64_t scales_s[3], scales_g;
  const float *gamma, *beta;
  float *dgamma, *dbeta, *ws;
};

// A row of the operands.
template <bool FLAT>
struct Row {
  uint32_t b, i, j;
  __device__ __forceinline__ Row(const Params& p, uint32_t r) {
    if (FLAT) {
      j = r;
      return;
    }
    const uint32_t q = quotient(p.n2, r);
    j = r - q * p.n2.d;
    b = quotient(p.n1, q);
    i = q - b * p.n1.d;
  }
  __device__ __forceinline__ int64_t at(const int64_t (&s)[3]) const {
    return FLAT ? (int64_t)j * s[2] : (int64_t)b * s[0] + (int64_t)i * s[1] + (int64_t)j * s[2];
  }
};

// The rows of group o (p.rows: there is none).
template <int T>
__device__ __forceinline__ void rows_of(const Params& p, uint32_t o, uint32_t (&r)[T]) {
  if (o >= p.groups) {
#pragma unroll
    for (int t = 0; t < T; ++t) r[t] = p.rows;
  } else if (p.along_i) {
    const uint32_t q = quotient(p.J, o), j = o - q * p.J.d, b = quotient(p.by_blocks_i, q),
                   i = (q - b * p.blocks_i) * T;
#pragma unroll
    for (int t = 0; t < T; ++t) r[t] = i + t < p.I.d ? (b * p.I.d + i + t) * p.J.d + j : p.rows;
  } else {
#pragma unroll
    for (int t = 0; t < T; ++t) r[t] = min(o * T + t, p.rows);
  }
}
__device__ __forceinline__ uint32_t mask_row(const Params& p, uint32_t r) {
  if (!p.shared) return r;
  const uint32_t q = quotient(p.J, r), b = quotient(p.I, q);
  return (uint32_t)(b * p.mask.s[0] + (q - b * p.I.d) * p.mask.s[1] + (r - q * p.J.d) * p.mask.s[2]);
}

// ---------------------------------------------------------------------------
// eight consecutive channels, or four that lie 32 apart, of either type
// ---------------------------------------------------------------------------
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen(float v) { return v; }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// What a load left, before it is widened: loads of a next row can be in flight
// at half the registers.
template <typename T, bool VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, true> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool ok) {
    a = ok ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw<float, true> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool ok) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    a = ok ? __ldcs(reinterpret_cast<const float4*>(p)) : z;
    b = ok ? __ldcs(reinterpret_cast<const float4*>(p) + 1) : z;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <typename T>
struct Raw<T, false> {
  T v[4];
  __device__ __forceinline__ void load(const T* p, int left) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = 32 * e < left ? p[32 * e] : narrow<T>(0.f);
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = widen(v[e]);
  }
};

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&f)[8], bool ok) {
  if (ok)
    *reinterpret_cast<uint4*>(p) = make_uint4(two_bf16(f[0], f[1]), two_bf16(f[2], f[3]),
                                              two_bf16(f[4], f[5]), two_bf16(f[6], f[7]));
}
__device__ __forceinline__ void put(float* p, const float (&f)[8], bool ok) {
  if (ok) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}
template <typename T>
__device__ __forceinline__ void put(T* p, const float (&f)[4], int left) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (32 * e < left) p[32 * e] = narrow<T>(f[e]);
}

// Where a thread's part of a row lies.
template <int LANES, bool VEC>
struct Lay {
  static constexpr int E = VEC ? 8 : 4;
  static constexpr int SPAN = VEC ? LANES * 8 : LANES * 4;  // channels of a part of the row
  // first channel of part k of thread `lane` of the row
  static __device__ __forceinline__ int chan(int lane, int k) {
    return VEC ? k * SPAN + lane * 8 : k * SPAN + (lane >> 5) * 128 + (lane & 31);
  }
    static __device__ __forceinline__ bool has(int C, int c, int e) { return VEC ? c < C : c + 32 * e < C; }
  static __device__ __forceinline__ int off(int e) { return VEC ? e : 32 * e; }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_part(Raw<T, VEC>& r, const void* base, int64_t at, int c, int C, bool on) {
  const T* p = static_cast<const T*>(base) + at + c;
  if constexpr (VEC)
    r.load(p, on && c < C);
  else
    r.load(p, on ? C - c : 0);
}
template <typename T, bool VEC, int E>
__device__ __forceinline__ void store_part(void* base, int64_t at, int c, int C, bool on, const float (&f)[E]) {
  T* p = static_cast<T*>(base) + at + c;
  if constexpr (VEC)
    put(p, f, on && c < C);
  else
    put(p, f, on ? C - c : 0);
}

// The factor of each element of a thread's part: 0 or 1 / (1 - p).
template <bool VEC, int E>
__device__ __forceinline__ void mask_factors(const PhiloxKey& key, const DropMask& m, int c, uint32_t row,
                                             float (&f)[E]) {
  if constexpr (VEC) {
    const uint32_t g = (uint32_t)c >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 w = philox(key, g + h, row);
      f[4 * h] = w.x >= m.threshold ? m.scale : 0.f;
      f[4 * h + 1] = w.y >= m.threshold ? m.scale : 0.f;
      f[4 * h + 2] = w.z >= m.threshold ? m.scale : 0.f;
      f[4 * h + 3] = w.w >= m.threshold ? m.scale : 0.f;
    }
  } else {
    // the warp's 128 channels are 32 blocks, one per lane; element e of this
    // lane is word lane % 4 of block 8 e + lane / 4
    const int lane = threadIdx.x & 31;
    const uint32_t mine = philox_keep4(key, m.threshold, ((uint32_t)(c - lane) >> 2) + lane, row);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = (__shfl_sync(0xffffffffu, mine, 8 * e + (lane >> 2)) >> (lane & 3) & 1u) ? m.scale : 0.f;
  }
}
// f * u, 0 where the factor is 0 whatever u is.
__device__ __forceinline__ float masked(float f, float u) { return f != 0.f ? f * u : 0.f; }

// Sums over the LANES threads of each of T rows, the same in all of them.  Rows
// wider than a warp go through shared memory: one barrier for the T of them, and
// `slot` differs between neighbouring calls.
template <int LANES, int T>
__device__ __forceinline__ void row_sums(float (&v)[T], float (*buf)[T][8], int slot) {
#pragma unroll
  for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int t = 0; t < T; ++t) v[t] += __shfl_xor_sync(0xffffffffu, v[t], o);
  if constexpr (LANES > 32) {
    constexpr int W = LANES / 32;
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int t = 0; t < T; ++t) buf[slot][t][warp] = v[t];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < T; ++t) {
      v[t] = buf[slot][t][first];
#pragma unroll
      for (int k = 1; k < W; ++k) v[t] += buf[slot][t][first + k];
    }
  }
}

constexpr int kThreads = 256;

// gamma or beta (1 or 0 where there is none, and beyond C) of all N channels that
// the threads of a row have places for, in shared memory.
template <int N>
__device__ __forceinline__ void load_params(float* to, const float* v, int C, float none) {
  for (int c = threadIdx.x; c < N; c += kThreads) to[c] = v && c < C ? v[c] : none;
}
__device__ __forceinline__ void get_params(const float* from, int c, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(from + c), b = *reinterpret_cast<const float4*>(from + c + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void get_params(const float* from, int c, float (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = from[c + 32 * e];
}

// Pairs of fp32.
__device__ __forceinline__ float2 pair(const float* f) { return make_float2(f[0], f[1]); }
__device__ __forceinline__ void put_pair(float* f, float2 v) { f[0] = v.x; f[1] = v.y; }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 1 / sqrt(v): the approximation with a Newton step, which leaves its own roundings
// (an error of y decides whether a maximum near the border between two scales
// takes the one or the other).  0 for an infinite v, as the approximation has it.
__device__ __forceinline__ float inverse_root(float v) {
  const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
  return fabsf(e) < 1.f ? fmaf(0.5f * r, e, r) : r;
}

// Rows minus their mean (layer norm), and 1 / sqrt(variance + eps).
template <int LANES, int PARTS, bool VEC, int T, int E>
__device__ __forceinline__ void centre(const Params& p, int lane, float (&x)[T][PARTS][E], float (&rstd)[T],
                                       float (*buf)[T][8]) {
  using L = Lay<LANES, VEC>;
  float mean[T];
#pragma unroll
  for (int t = 0; t < T; ++t) mean[t] = 0.f;
  if (!p.rms) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float2 s = both(0.f);
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
#pragma unroll
        for (int e = 0; e < E; e += 2) s = add2(s, pair(&x[t][k][e]));
      mean[t] = s.x + s.y;
    }
    row_sums<LANES, T>(mean, buf, 0);
#pragma unroll
    for (int t = 0; t < T; ++t) mean[t] *= p.inv_c;
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    float2 s = both(0.f);
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 m = make_float2(L::has(p.C, c, e) ? -mean[t] : 0.f, L::has(p.C, c, e + 1) ? -mean[t] : 0.f);
        const float2 d = add2(pair(&x[t][k][e]), m);
        put_pair(&x[t][k][e], d);
        s = fma2(d, d, s);
      }
    }
    rstd[t] = s.x + s.y;
  }
  row_sums<LANES, T>(rstd, buf, 1);
#pragma unroll
  for (int t = 0; t < T; ++t) rstd[t] = inverse_root(rstd[t] * p.inv_c + p.eps);
}

// ---------------------------------------------------------------------------
// dropout and residual add
// ---------------------------------------------------------------------------
// A thread takes one part of each of T rows; nothing is shared between threads.
template <typename S, typename IO, bool VEC, bool FLAT, int T>
__global__ void __launch_bounds__(kThreads) k_dropout_add(const Params p, Divide parts, uint32_t items) {
  wait_for_earlier_work();
  let_next_start();
  PhiloxKey key{};
  if (p.drop) key = philox_key(p.mask);
  constexpr int E = VEC ? 8 : 4;
  const uint32_t id = VEC ? blockIdx.x * kThreads + threadIdx.x : blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (id >= items) return;  // (whole warps, where a warp works together)
  const uint32_t o = quotient(parts, id), part = id - o * parts.d;
  const int c = VEC ? (int)part * 8 : (int)part * 128 + (threadIdx.x & 31);
  uint32_t r[T];
  rows_of<T>(p, o, r);
  Raw<IO, VEC> ru[T];
  Raw<S, VEC> rx[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const bool on = r[t] < p.rows;
    const Row<FLAT> w(p, on ? r[t] : 0);
    load_part<IO, VEC>(ru[t], p.u.p, w.at(p.u.s), c, p.C, on);
    if (p.x.p) load_part<S, VEC>(rx[t], p.x.p, w.at(p.x.s), c, p.C, on);
  }
  float m[E];
#pragma unroll
  for (int e = 0; e < E; ++e) m[e] = 1.f;
  uint32_t drawn = 0xFFFFFFFFu;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const bool on = r[t] < p.rows;
    const Row<FLAT> w(p, on ? r[t] : 0);
    float f[E], x[E];
    ru[t].get(f);
    if (p.drop) {
      const uint32_t row = mask_row(p, on ? r[t] : 0);
      if (row != drawn) mask_factors<VEC>(key, p.mask, c, row, m);
      drawn = row;
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = masked(m[e], f[e]);
    }
    if (p.x.p) {
      rx[t].get(x);
#pragma unroll
      for (int e = 0; e < E; e += 2) put_pair(&f[e], add2(pair(&f[e]), pair(&x[e])));
    }
    store_part<S, VEC>(p.x1.p, w.at(p.x1.s), c, p.C, on, f);
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename S, typename IO, int LANES, int PARTS, bool VEC, bool FLAT, int T>
__global__ void __launch_bounds__(kThreads, VEC && FLAT && PARTS == 1 && sizeof(S) == 2 ? 4 : 3) k_norm8_fwd(const Params p, uint32_t turns) {
  using L = Lay<LANES, VEC>;
  constexpr int E = L::E, PER = kThreads / LANES;
  __shared__ float sums[2][T][8];
  constexpr int N = PARTS * L::SPAN;  // channels that the threads of a row have places for
  __shared__ __align__(16) float prm[2 * N];  // gamma, beta
  float* const prm_b = prm + N;
  wait_for_earlier_work();
  let_next_start();
  const int lane = threadIdx.x % LANES;
  PhiloxKey key{};
  if (p.drop) key = philox_key(p.mask);
  // (a loop only where a CTA takes several turns: it costs registers)
  const uint32_t mine = LANES > 64 ? turns : 1;
#pragma unroll 1
  for (uint32_t turn = 0; turn < mine; ++turn) {
    uint32_t r[T];
    rows_of<T>(p, (blockIdx.x * mine + turn) * PER + threadIdx.x / LANES, r);
    Raw<S, VEC> rx[T][PARTS];
    Raw<IO, VEC> ru[T][PARTS];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const bool on = r[t] < p.rows;
      const Row<FLAT> w(p, on ? r[t] : 0);
      const int64_t ax = w.at(p.x.s), au = w.at(p.u.s);
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        load_part<S, VEC>(rx[t][k], p.x.p, ax, L::chan(lane, k), p.C, on);
        if (p.u.p) load_part<IO, VEC>(ru[t][k], p.u.p, au, L::chan(lane, k), p.C, on);
      }
    }
    if (turn == 0) {
      load_params<N>(prm, p.gamma, p.C, 1.f);
      load_params<N>(prm_b, p.beta, p.C, 0.f);
      __syncthreads();
    } else if (LANES > 64) {
      __syncthreads();  // the sums of the turn before
    }
    float x[T][PARTS][E];
    if (p.u.p) {
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const int c = L::chan(lane, k);
        float m[E];
#pragma unroll
        for (int e = 0; e < E; ++e) m[e] = 1.f;
        uint32_t drawn = 0xFFFFFFFFu;
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const bool on = r[t] < p.rows;
          float f[E];
          ru[t][k].get(f);
          if (p.drop) {
            const uint32_t row = mask_row(p, on ? r[t] : 0);
            if (row != drawn) mask_factors<VEC>(key, p.mask, c, row, m);
            drawn = row;
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = masked(m[e], f[e]);
          }
          rx[t][k].get(x[t][k]);
#pragma unroll
          for (int e = 0; e < E; e += 2) put_pair(&x[t][k][e], add2(pair(&x[t][k][e]), pair(&f[e])));
          const Row<FLAT> w(p, on ? r[t] : 0);
          store_part<S, VEC>(p.x1.p, w.at(p.x1.s), c, p.C, on, x[t][k]);
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int k = 0; k < PARTS; ++k) rx[t][k].get(x[t][k]);
    }
    float rstd[T];
    centre<LANES, PARTS, VEC, T, E>(p, lane, x, rstd, sums);
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
      float ga[E], be[E];
      get_params(prm, c, ga);
      get_params(prm_b, c, be);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const bool on = r[t] < p.rows;
        const Row<FLAT> w(p, on ? r[t] : 0);
        float(&y)[E] = x[t][k];
#pragma unroll
        for (int e = 0; e < E; e += 2)
          put_pair(&y[e], fma2(mul2(pair(&y[e]), both(rstd[t])), pair(&ga[e]), pair(&be[e])));
        if (!VEC) {
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = L::has(p.C, c, e) ? y[e] : 0.f;
        }
        const auto group_maximum = [&] {
          float m = max_abs(y);
#pragma unroll
          for (int o = (VEC ? (LANES < 16 ? LANES : 16) : 32) / 2; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          return m;
        };
        if (VEC && c >= p.C) {  // (beta of a part beyond the row is 0, and so is y)
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = 0.f;
        }
        float amax = group_maximum();
        if (__any_sync(0xffffffffu, amax > FLT_MAX)) {
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = infinity_to_nan(y[e]);
          amax = group_maximum();
        }
        const uint32_t code = scale_code(amax);
        const float inv = scale_inverse(code);
        const int64_t ac = w.at(p.codes_s);
        if constexpr (VEC) {
          if (on && c < p.C)
            *reinterpret_cast<uint2*>(p.codes + ac + c) =
                make_uint2(e4m3_four(y[0], y[1], y[2], y[3], inv), e4m3_four(y[4], y[5], y[6], y[7], inv));
        } else {
          const uint32_t q = e4m3_four(y[0], y[1], y[2], y[3], inv);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (on && c + 32 * e < p.C) p.codes[ac + c + 32 * e] = (uint8_t)(q >> 8 * e);
        }
        if (on && (c & 127) == 0 && c < p.C)
          p.scales[w.at(p.scales_s) + (int64_t)(c >> 7) * p.scales_g] = (uint8_t)code;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Persistent: a thread adds the parameter gradients of its channels over all
// its rows in registers, a CTA adds its row groups in order and leaves one
// partial sum, and a second kernel adds those in order.
//
// The sums hold 128 registers and with them 16 warps per SM, too few to cover the
// memory's latency with loads into registers (58 us for 147,456 bf16 rows of 128
// where the bytes take 28).  Whole 16-byte units therefore come through a ring of
// DEPTH turns in shared memory, filled by cp.async: a thread copies, and reads,
// only its own units, so the ring needs no barrier.  A thread's fp32 part is two
// units, which its neighbours' lie between: they go through L1, which keeps the other
// half of a 32-byte sector (195,330 rows of 72 with an fp32 stream 58 -> 51 us, past L1
// 70).  Rows that are fp32 throughout are loaded into registers (108 us for 262,144
// of 128, 91 % of the copy rate).
template <typename S, typename IO, int PARTS, int T>
struct Ring {
  static constexpr int UNITS_S = sizeof(S) / 2, UNITS_IO = sizeof(IO) / 2;  // of 16 bytes, for 8 elements
  static constexpr int UNITS = T * PARTS * (2 * UNITS_S + UNITS_IO);        // of a thread's turn: x1, dx1, dy
  static constexpr uint32_t STAGE = UNITS * kThreads * 16;
  static constexpr int DEPTH = std::min<int>(4, std::max<int>(2, (int)(80 * 1024 / STAGE)));
  static constexpr bool USED = sizeof(IO) == 2;
  static constexpr uint32_t BYTES = DEPTH * STAGE;
};
// (a unit of which nothing is read is zero)
template <bool WHOLE>
__device__ __forceinline__ void copy_unit(uint32_t to, const void* from, bool on) {
  if constexpr (WHOLE)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
template <typename T>
__device__ __forceinline__ void copy_part(uint32_t to, const void* base, int64_t at, int c, bool on) {
  const T* p = static_cast<const T*>(base) + (on ? at + c : 0);
#pragma unroll
  for (int u = 0; u < (int)sizeof(T) / 2; ++u) copy_unit<sizeof(T) == 2>(to + u * kThreads * 16, p + u * 16 / sizeof(T), on);
}
template <typename T>
__device__ __forceinline__ void read_part(const uint4* from, Raw<T, true>& r) {
  if constexpr (sizeof(T) == 2) {
    r.a = from[0];
  } else {
    r.a = *reinterpret_cast<const float4*>(from);
    r.b = *reinterpret_cast<const float4*>(from + kThreads);
  }
}

template <typename S, typename IO, int LANES, int PARTS, bool VEC, bool FLAT, int T>
__global__ void __launch_bounds__(kThreads, 2) k_norm8_bwd(const Params p, uint32_t turns) {
  using L = Lay<LANES, VEC>;
  constexpr int E = L::E, PER = kThreads / LANES;
  __shared__ float sums[2][T][8], sums2[2][T][8];
  constexpr int N = PARTS * L::SPAN;  // channels that the threads of a row have places for (C at least)
  __shared__ __align__(16) float prm[N];  // gamma
  wait_for_earlier_work();
  let_next_start();
  const int lane = threadIdx.x % LANES;
  load_params<N>(prm, p.gamma, p.C, 1.f);
  PhiloxKey key{};
  if (p.drop) key = philox_key(p.mask);
  __syncthreads();
  float ag[PARTS][E], ab[PARTS][E];
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) ag[k][e] = ab[k][e] = 0.f;
  using R = Ring<S, IO, PARTS, T>;
  extern __shared__ __align__(16) uint4 ring[];
  const auto rows_at = [&](uint32_t turn, uint32_t (&r)[T]) {
    rows_of<T>(p, (turn * gridDim.x + blockIdx.x) * PER + threadIdx.x / LANES, r);
  };
  // this thread's units of a turn into its slots
  const auto fill = [&](uint32_t turn) {
    if (turn < turns) {
      uint32_t r[T];
      rows_at(turn, r);
      uint32_t to = smem_u32(ring) + (turn % R::DEPTH) * R::STAGE + threadIdx.x * 16;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const bool on = r[t] < p.rows;
        const Row<FLAT> w(p, on ? r[t] : 0);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          const int c = L::chan(lane, k);
          copy_part<S>(to, p.x1.p, w.at(p.x1.s), c, on && c < p.C);
          if (p.dx1.p) copy_part<S>(to + R::UNITS_S * kThreads * 16, p.dx1.p, w.at(p.dx1.s), c, on && c < p.C);
          copy_part<IO>(to + 2 * R::UNITS_S * kThreads * 16, p.dy.p, w.at(p.dy.s), c, on && c < p.C);
          to += (2 * R::UNITS_S + R::UNITS_IO) * kThreads * 16;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (VEC && R::USED) {
#pragma unroll
    for (int k = 0; k < R::DEPTH - 1; ++k) fill(k);
  }
#pragma unroll 1
  for (uint32_t turn = 0; turn < turns; ++turn) {
    uint32_t r[T];
    rows_at(turn, r);
    Raw<S, VEC> rx[T][PARTS], rd[T][PARTS];
    Raw<IO, VEC> ry[T][PARTS];
    if constexpr (VEC && R::USED) {
      fill(turn + R::DEPTH - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(R::DEPTH - 1) : "memory");
      const uint4* from = ring + (turn % R::DEPTH) * (R::STAGE / 16) + threadIdx.x;
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          read_part<S>(from, rx[t][k]);
          if (p.dx1.p) read_part<S>(from + R::UNITS_S * kThreads, rd[t][k]);
          read_part<IO>(from + 2 * R::UNITS_S * kThreads, ry[t][k]);
          from += (2 * R::UNITS_S + R::UNITS_IO) * kThreads;
        }
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const bool on = r[t] < p.rows;
        const Row<FLAT> w(p, on ? r[t] : 0);
        const int64_t ax = w.at(p.x1.s), ad = w.at(p.dx1.s), ay = w.at(p.dy.s);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          const int c = L::chan(lane, k);
          load_part<S, VEC>(rx[t][k], p.x1.p, ax, c, p.C, on);
          load_part<IO, VEC>(ry[t][k], p.dy.p, ay, c, p.C, on);
          if (p.dx1.p) load_part<S, VEC>(rd[t][k], p.dx1.p, ad, c, p.C, on);
        }
      }
    }
    float h[T][PARTS][E], rstd[T], m1[T], m2[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int k = 0; k < PARTS; ++k) rx[t][k].get(h[t][k]);
    centre<LANES, PARTS, VEC, T, E>(p, lane, h, rstd, sums);
    float g[T][PARTS][E];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        ry[t][k].get(g[t][k]);
        float ga[E];
        get_params(prm, L::chan(lane, k), ga);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 hh = mul2(pair(&h[t][k][e]), both(rstd[t])), gg = pair(&g[t][k][e]);
          put_pair(&h[t][k][e], hh);
          put_pair(&ag[k][e], fma2(gg, hh, pair(&ag[k][e])));
          put_pair(&ab[k][e], add2(gg, pair(&ab[k][e])));
          const float2 ee = mul2(gg, pair(&ga[e]));
          put_pair(&g[t][k][e], ee);
          s1 = fma2(ee, hh, s1);
          s2 = add2(ee, s2);
        }
      }
      m1[t] = s1.x + s1.y;
      m2[t] = s2.x + s2.y;
    }
    row_sums<LANES, T>(m1, sums2, 0);
    if (!p.rms) row_sums<LANES, T>(m2, sums2, 1);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      m1[t] *= -p.inv_c;
      m2[t] = p.rms ? 0.f : m2[t] * -p.inv_c;
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
      float m[E];
      uint32_t drawn = 0xFFFFFFFFu;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const bool on = r[t] < p.rows;
        const Row<FLAT> w(p, on ? r[t] : 0);
        float d[E];
        if (p.dx1.p) {
          rd[t][k].get(d);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = fma2(pair(&h[t][k][e]), both(m1[t]), add2(pair(&g[t][k][e]), both(m2[t])));
          put_pair(&d[e], fma2(both(rstd[t]), v, pair(&d[e])));
        }
        store_part<S, VEC>(p.dx.p, w.at(p.dx.s), c, p.C, on, d);
        if (p.du.p) {
          if (p.drop) {
            const uint32_t row = mask_row(p, on ? r[t] : 0);
            if (row != drawn) mask_factors<VEC>(key, p.mask, c, row, m);
            drawn = row;
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = masked(m[e], d[e]);
          }
          store_part<IO, VEC>(p.du.p, w.at(p.du.s), c, p.C, on, d);
        }
      }
    }
    if constexpr (LANES > 32) __syncthreads();  // the next rows' sums
  }
  // The CTA's sums: a warp's row groups by shuffles, then each warp's sums lie in
  // shared memory and are added in order.
  constexpr int ROWS = LANES <= 32 ? kThreads / 32 : PER;  // sums of a channel that are left
  float* const sums_g = reinterpret_cast<float*>(ring);
  if constexpr (VEC && R::USED) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();  // (every thread is through with the ring)
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float g = ag[k][e], b = ab[k][e];
#pragma unroll
      for (int o = 16; o >= LANES; o >>= 1) {
        g += __shfl_xor_sync(0xffffffffu, g, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      const int row = LANES <= 32 ? (int)threadIdx.x >> 5 : (int)threadIdx.x / LANES;
      if (LANES >= 32 || (int)(threadIdx.x & 31) < LANES) {
        float* to = sums_g + row * 2 * N + L::chan(lane, k) + L::off(e);
        to[0] = g;
        to[N] = b;
      }
    }
  __syncthreads();
  float* out = p.ws + (int64_t)blockIdx.x * 2 * p.C;
  for (int c = threadIdx.x; c < 2 * p.C; c += kThreads) {
    const float* from = sums_g + (c < p.C ? c : N + c - p.C);
    float v = from[0];
#pragma unroll
    for (int q = 1; q < ROWS; ++q) v += from[q * 2 * N];
    out[c] = v;
  }
}

// Partial sums of `count` CTAs: 32 warps share 32 columns, each a stretch of the
// CTAs (19 at most, so one or two rounds of loads), joined in a fixed order.
template <typename S>
__global__ void __launch_bounds__(1024) k_norm8_reduce(const Params p, int count) {
  __shared__ float buf[32][33];
  wait_for_earlier_work();
  let_next_start();
  const int warp = threadIdx.x >> 5, c = blockIdx.x * 32 + (threadIdx.x & 31);
  const int per = (count + 31) / 32, lo = warp * per, hi = min(count, lo + per);
  float s = 0.f;
  if (c < 2 * p.C)
#pragma unroll 10
    for (int k = lo; k < hi; ++k) s += p.ws[(int64_t)k * 2 * p.C + c];
  buf[warp][threadIdx.x & 31] = s;
  __syncthreads();
  // warp w adds column w's stretches
  s = buf[threadIdx.x & 31][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + warp;
  if ((threadIdx.x & 31) == 0 && col < 2 * p.C) {
    float* out = col < p.C ? p.dgamma : p.dbeta;
    if (out) out[col < p.C ? col : col - p.C] = s;
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
inline bool aligned16(const RowOperand& o, size_t size) {
  if (!o.p) return true;
  if (reinterpret_cast<uintptr_t>(o.p) % 16) return false;
  for (int64_t s : o.s)
    if (s * (int64_t)size % 16) return false;
  return true;
}

inline Params params_of(const Norm8Call& c, int T) {
  Params p{};
  p.rows = (uint32_t)c.n[0] * (uint32_t)c.n[1] * (uint32_t)c.n[2];
  p.n1 = divide_by((uint32_t)c.n[1]);
  p.n2 = divide_by((uint32_t)c.n[2]);
  p.I = divide_by((uint32_t)c.given[1]);
  p.J = divide_by((uint32_t)c.given[2]);
  const auto shares = [&](int k) { return c.drop && c.given[k] > 1 && c.mask.s[k] == 0; };
  p.shared = c.drop && (c.turned || shares(0) || shares(1) || shares(2));
  p.along_i = shares(1) && !shares(2);
  p.blocks_i = (uint32_t)(c.given[1] + T - 1) / T;
  p.by_blocks_i = divide_by(p.blocks_i);
  p.groups = p.along_i ? (uint32_t)c.given[0] * p.blocks_i * (uint32_t)c.given[2] : (p.rows + T - 1) / T;
  p.C = c.C;
  p.inv_c = 1.0f / (float)c.C;
  p.eps = c.eps;
  p.rms = c.rms;
  p.drop = c.drop;
  p.mask = c.mask;
  p.x = c.x; p.u = c.u; p.x1 = c.x1;
  p.dx1 = c.dx1; p.dy = c.dy; p.dx = c.dx; p.du = c.du;
  p.codes = c.codes; p.scales = c.scales; p.scales_g = c.scales_g;
  for (int k = 0; k < 3; ++k) { p.codes_s[k] = c.codes_s[k]; p.scales_s[k] = c.scales_s[k]; }
  p.gamma = c.gamma; p.beta = c.beta;
  p.dgamma = c.dgamma; p.dbeta = c.dbeta; p.ws = c.ws;
  return p;
}

// Calls f(std::integral_constant<bool, v>).
template <typename F>
cudaError_t by_flag(bool v, F&& f) {
  return v ? f(std::integral_constant<bool, true>{}) : f(std::integral_constant<bool, false>{});
}

template <typename S, typename IO>
cudaError_t run_dropout(const Norm8Call& c, cudaStream_t st) {
  constexpr int T = 4;
  const Params p = params_of(c, T);
  const bool vec = c.C % 8 == 0 && aligned16(c.x, sizeof(S)) && aligned16(c.x1, sizeof(S)) &&
                   aligned16(c.u, sizeof(IO));
  const uint32_t parts = vec ? (uint32_t)c.C / 8 : (uint32_t)(c.C + 127) / 128;
  // (a part's index takes 31 bits)
  const uint64_t items = (uint64_t)p.groups * parts, per_cta = vec ? kThreads : kThreads / 32;
  if (items > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)((items + per_cta - 1) / per_cta);
  return by_flag(vec, [&](auto v) {
    return by_flag(c.n[0] == 1 && c.n[1] == 1, [&](auto flat) {
      return launch_early(k_dropout_add<S, IO, decltype(v)::value, decltype(flat)::value, T>, grid, kThreads, 0, st, p,
                          divide_by(parts), (uint32_t)items);
    });
  });
}

// The threads of a row, its parts per thread and the rows that a thread holds, by
// the channel count: 16 channels of a row per thread at most, in the forward 24
// where that fits 384 or 768 exactly (THREE; the backward's sums leave no registers
// for it), so that four rows' (or two's) operands stay in registers.
template <bool VEC, bool THREE, typename F>
cudaError_t by_width(int C, F&& f) {
#define EVO_N8(lanes, parts, rows) \
  return f(std::integral_constant<int, lanes>{}, std::integral_constant<int, parts>{}, std::integral_constant<int, rows>{})
  if constexpr (VEC) {
    if (C <= 64) EVO_N8(8, 1, 4);
    if (C <= 128) EVO_N8(16, 1, 4);
    if (C <= 256) EVO_N8(32, 1, 4);
    if constexpr (THREE) {
      if (C <= 384) EVO_N8(16, 3, 2);
    }
    if (C <= 512) EVO_N8(32, 2, 2);
    if constexpr (THREE) {
      if (C <= 768) EVO_N8(32, 3, 2);
    }
    if (C <= 1024) EVO_N8(64, 2, 2);
    if (C <= 2048) EVO_N8(128, 2, 2);
    EVO_N8(256, 2, 2);
  } else {
    if (C <= 128) EVO_N8(32, 1, 4);
    if (C <= 256) EVO_N8(32, 2, 4);
    if (C <= 512) EVO_N8(32, 4, 2);
    if (C <= 1024) EVO_N8(64, 4, 2);
    if (C <= 2048) EVO_N8(128, 4, 2);
    EVO_N8(256, 4, 2);
  }
#undef EVO_N8
}

template <typename S, typename IO, bool VEC>
cudaError_t run_fwd_as(const Norm8Call& c, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return by_width<VEC, true>(c.C, [&](auto lanes, auto parts, auto rows) {
    constexpr int L = decltype(lanes)::value, P = decltype(parts)::value, T = decltype(rows)::value;
    constexpr uint32_t per = kThreads / L;
    static_assert(2 * P * Lay<L, VEC>::SPAN * sizeof(float) <= 32 * 1024, "static shared memory");
    const Params p = params_of(c, T);
    return by_flag(c.n[0] == 1 && c.n[1] == 1, [&](auto flat) {
      // Short CTAs; but a wide row's gamma and beta are read again by every CTA,
      // so there four turns share them, as long as there are CTAs enough.
      const uint32_t ctas = (p.groups + per - 1) / per;
      const uint32_t turns = L <= 64 ? 1 : std::min<uint32_t>(4, std::max<uint32_t>(1, ctas / (6 * sms)));
      return launch_early(k_norm8_fwd<S, IO, L, P, VEC, decltype(flat)::value, T>, (ctas + turns - 1) / turns, kThreads,
                          0, st, p, turns);
    });
  });
}

template <typename S, typename IO>
cudaError_t run_fwd(const Norm8Call& c, cudaStream_t st) {
  bool vec = c.C % 8 == 0 && aligned16(c.x, sizeof(S)) && aligned16(c.x1, sizeof(S)) &&
             aligned16(c.u, sizeof(IO)) && reinterpret_cast<uintptr_t>(c.codes) % 8 == 0;
  for (int64_t s : c.codes_s) vec = vec && s % 8 == 0;
  return vec ? run_fwd_as<S, IO, true>(c, st) : run_fwd_as<S, IO, false>(c, st);
}

template <typename S, typename IO, bool VEC>
cudaError_t run_bwd_as(const Norm8Call& c, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return by_width<VEC, false>(c.C, [&](auto lanes, auto parts, auto rows) {
    constexpr int L = decltype(lanes)::value, P = decltype(parts)::value, T = decltype(rows)::value / 2;
    constexpr uint32_t per = kThreads / L;
    const Params p = params_of(c, T);
    const cudaError_t e2 = by_flag(c.n[0] == 1 && c.n[1] == 1, [&](auto flat) {
      auto kern = k_norm8_bwd<S, IO, L, P, VEC, decltype(flat)::value, T>;
      // the ring, and in the end the sums of gamma and beta of eight warps
      constexpr size_t sums = (size_t)(L <= 32 ? kThreads / 32 : kThreads / L) * 2 * P * Lay<L, VEC>::SPAN * sizeof(float);
      constexpr size_t smem = std::max<size_t>(VEC && Ring<S, IO, P, T>::USED ? Ring<S, IO, P, T>::BYTES : 0, sums);
      cudaError_t e3 = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e3 != cudaSuccess) return e3;
      // CTAs that an SM holds (asked once per device: a property of the kernel)
      static std::atomic<int> held[64];
      int fit = dev < 64 ? held[dev].load() : 0;
      if (fit == 0) {
        e3 = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, kThreads, smem);
        if (e3 != cudaSuccess) return e3;
        if (dev < 64) held[dev].store(fit);
      }
      const uint32_t want = (p.groups + per - 1) / per;
      const uint32_t most = std::min<uint32_t>(kNorm8MaxCtas, (uint32_t)std::max(1, fit * sms));
      const uint32_t turns = (want + most - 1) / most;
      const uint32_t grid = (want + turns - 1) / turns;
      e3 = launch_early(kern, grid, kThreads, smem, st, p, turns);
      if (e3 != cudaSuccess || (!p.dgamma && !p.dbeta)) return e3;
      return launch_early(k_norm8_reduce<S>, (unsigned)(2 * c.C + 31) / 32, 1024, 0, st, p, (int)grid);
    });
    return e2;
  });
}

template <typename S, typename IO>
cudaError_t run_bwd(const Norm8Call& c, cudaStream_t st) {
  const bool vec = c.C % 8 == 0 && aligned16(c.x1, sizeof(S)) && aligned16(c.dx1, sizeof(S)) &&
                   aligned16(c.dx, sizeof(S)) && aligned16(c.dy, sizeof(IO)) && aligned16(c.du, sizeof(IO));
  return vec ? run_bwd_as<S, IO, true>(c, st) : run_bwd_as<S, IO, false>(c, st);
}

}  // namespace norm8
}  // namespace evo
