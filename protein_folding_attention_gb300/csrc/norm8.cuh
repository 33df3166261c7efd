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
// wherever it is needed (philox.cuh).
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

#include "launch.cuh"
#include "norm8.h"
#include "philox.cuh"
#include "scale8.cuh"

namespace evo {
namespace norm8 {

struct Params {
  uint32_t rows;
  uint32_t n1, n2;  // row r = (b * n1 + i) * n2 + j
  int C, groups;
  float inv_c, eps;
  bool rms;
  DropMask mask;
  RowOperand x, u, x1, dx1, dy, dx, du;
  uint8_t* codes;
  int64_t codes_s[3];
  uint8_t* scales;
  int64_t scales_s[3], scales_g;
  const float *gamma, *beta;
  float *dgamma, *dbeta, *ws;
};

struct Row {
  uint32_t b, i, j;
  __device__ __forceinline__ int64_t at(const int64_t (&s)[3]) const {
    return (int64_t)b * s[0] + (int64_t)i * s[1] + (int64_t)j * s[2];
  }
};
__device__ __forceinline__ Row row_of(const Params& p, uint32_t r) {
  Row w;
  const uint32_t q = p.n2 == 1 ? r : r / p.n2;
  w.j = r - q * p.n2;
  w.b = p.n1 == 1 ? q : q / p.n1;
  w.i = q - w.b * p.n1;
  return w;
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
  // channels from there on (VEC: as a truth value, parts are whole)
  static __device__ __forceinline__ int left(int C, int c) { return C - c; }
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

// Keep bits of a thread's part (bit e: element e).
template <bool VEC>
__device__ __forceinline__ uint32_t keep_bits(const PhiloxKey& key, uint32_t threshold, int c, uint32_t row) {
  if constexpr (VEC) {
    const uint32_t g = (uint32_t)c >> 2;
    return philox_keep4(key, threshold, g, row) | philox_keep4(key, threshold, g + 1, row) << 4;
  } else {
    // the warp's 128 channels are 32 blocks, one per lane; element e of this
    // lane is word lane % 4 of block 8 e + lane / 4
    const int lane = threadIdx.x & 31;
    const uint32_t mine = philox_keep4(key, threshold, ((uint32_t)(c - lane) >> 2) + lane, row);
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      bits |= (__shfl_sync(0xffffffffu, mine, 8 * e + (lane >> 2)) >> (lane & 3) & 1u) << e;
    return bits;
  }
}

// Sum over the LANES threads of a row, the same in all of them.  Rows wider than
// a warp go through shared memory; `slot` alternates between calls.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float (*buf)[32], int slot) {
#pragma unroll
  for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (LANES > 32) {
    constexpr int W = LANES / 32;
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0) buf[slot][warp] = v;
    __syncthreads();
    v = buf[slot][first];
#pragma unroll
    for (int k = 1; k < W; ++k) v += buf[slot][first + k];
  }
  return v;
}

// ---------------------------------------------------------------------------
// dropout and residual add
// ---------------------------------------------------------------------------
// Threads of a warp take consecutive parts of consecutive rows; nothing is
// shared between them.
template <typename S, typename IO, bool VEC>
__global__ void __launch_bounds__(256) k_dropout_add(const Params p, uint64_t items, uint32_t per_row, bool drop) {
  wait_for_earlier_work();
  let_next_start();
  PhiloxKey key{};
  if (drop) key = philox_key(p.mask);
  const uint64_t id = (uint64_t)blockIdx.x * (VEC ? 256 : 8) + (VEC ? threadIdx.x : threadIdx.x >> 5);
  const bool on = id < items;
  const uint32_t r = on ? ((items >> 32) ? (uint32_t)(id / per_row) : (uint32_t)id / per_row) : 0;
  const int at = on ? (int)(id - (uint64_t)r * per_row) : 0;
  const int c = VEC ? at * 8 : at * 128 + (threadIdx.x & 31);
  constexpr int E = VEC ? 8 : 4;
  const Row w = row_of(p, r);
  Raw<IO, VEC> ru;
  Raw<S, VEC> rx;
  load_part<IO, VEC>(ru, p.u.p, w.at(p.u.s), c, p.C, on);
  if (p.x.p) load_part<S, VEC>(rx, p.x.p, w.at(p.x.s), c, p.C, on);
  float f[E], x[E];
  ru.get(f);
  if (drop) {
    const uint32_t bits = keep_bits<VEC>(key, p.mask.threshold, c, (uint32_t)w.at(p.mask.s));
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = (bits >> e & 1) ? f[e] * p.mask.scale : 0.f;
  }
  if (p.x.p) {
    rx.get(x);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] += x[e];
  }
  store_part<S, VEC>(p.x1.p, w.at(p.x1.s), c, p.C, on, f);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
constexpr int kThreads = 128;

template <typename S, typename IO, int LANES, int PARTS, bool VEC>
__global__ void __launch_bounds__(kThreads) k_norm8_fwd(const Params p, int turns, bool drop) {
  using L = Lay<LANES, VEC>;
  constexpr int E = L::E, PER = kThreads / LANES;
  __shared__ float sums[2][32];
  wait_for_earlier_work();
  let_next_start();
  const int lane = threadIdx.x % LANES;
  PhiloxKey key{};
  if (drop) key = philox_key(p.mask);
  uint32_t r = (uint32_t)blockIdx.x * (uint32_t)(PER * turns) + threadIdx.x / LANES;
#pragma unroll 1
  for (int t = 0; t < turns; ++t, r += PER) {
    if (r - threadIdx.x / LANES >= p.rows) break;  // (the same for the whole CTA)
    const bool on = r < p.rows;
    const Row w = row_of(p, on ? r : 0);
    Raw<S, VEC> rx[PARTS];
    Raw<IO, VEC> ru[PARTS];
    const int64_t ax = w.at(p.x.s), au = w.at(p.u.s);
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      load_part<S, VEC>(rx[k], p.x.p, ax, L::chan(lane, k), p.C, on);
      if (p.u.p) load_part<IO, VEC>(ru[k], p.u.p, au, L::chan(lane, k), p.C, on);
    }
    float x[PARTS][E];
    float sum = 0.f;
    const uint32_t mrow = drop ? (uint32_t)w.at(p.mask.s) : 0u;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
      rx[k].get(x[k]);
      if (p.u.p) {
        float f[E];
        ru[k].get(f);
        if (drop) {
          const uint32_t bits = keep_bits<VEC>(key, p.mask.threshold, c, mrow);
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = (bits >> e & 1) ? f[e] * p.mask.scale : 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] += f[e];
        store_part<S, VEC>(p.x1.p, w.at(p.x1.s), c, p.C, on, x[k]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum += x[k][e];
    }
    float mean = 0.f;
    if (!p.rms) mean = row_sum<LANES>(sum, sums, 0) * p.inv_c;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = L::has(p.C, L::chan(lane, k), e) ? x[k][e] - mean : 0.f;
        x[k][e] = d;
        sq = fmaf(d, d, sq);
      }
    const float rstd = rsqrtf(row_sum<LANES>(sq, sums, 1) * p.inv_c + p.eps);
    const int64_t ac = w.at(p.codes_s), as = w.at(p.scales_s);
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool has = L::has(p.C, c, e);
        float y = x[k][e] * rstd;
        if (has && p.gamma) y *= p.gamma[c + L::off(e)];
        if (has && p.beta) y += p.beta[c + L::off(e)];
        x[k][e] = y;
      }
      const auto group_maximum = [&] {
        float m = max_abs(x[k]);
#pragma unroll
        for (int o = (VEC ? (LANES < 16 ? LANES : 16) : 32) / 2; o > 0; o >>= 1)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
      };
      float amax = group_maximum();
      if (__any_sync(0xffffffffu, amax > FLT_MAX)) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] = infinity_to_nan(x[k][e]);
        amax = group_maximum();
      }
      const uint32_t code = scale_code(amax);
      const float inv = scale_inverse(code);
      if constexpr (VEC) {
        const uint2 q = make_uint2(e4m3_four(x[k][0], x[k][1], x[k][2], x[k][3], inv),
                                   e4m3_four(x[k][4], x[k][5], x[k][6], x[k][7], inv));
        if (on && c < p.C) {
          *reinterpret_cast<uint2*>(p.codes + ac + c) = q;
          if ((c & 127) == 0) p.scales[as + (int64_t)(c >> 7) * p.scales_g] = (uint8_t)code;
        }
      } else {
        const uint32_t q = e4m3_four(x[k][0], x[k][1], x[k][2], x[k][3], inv);
        if (on) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + 32 * e < p.C) p.codes[ac + c + 32 * e] = (uint8_t)(q >> 8 * e);
          if ((c & 127) == 0 && c < p.C) p.scales[as + (int64_t)(c >> 7) * p.scales_g] = (uint8_t)code;
        }
      }
    }
    if constexpr (LANES > 32) __syncthreads();  // the next row's sums
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Persistent: a thread adds the parameter gradients of its channels over all
// its rows in registers, a CTA adds its row groups in order and leaves one
// partial sum, and a second kernel adds those in order.
template <typename S, typename IO, int LANES, int PARTS, bool VEC>
__global__ void __launch_bounds__(kThreads) k_norm8_bwd(const Params p, uint32_t turns, bool drop) {
  using L = Lay<LANES, VEC>;
  constexpr int E = L::E, PER = kThreads / LANES;
  __shared__ float sums[4][32];
  extern __shared__ float part[];  // [2][C]
  wait_for_earlier_work();
  let_next_start();
  const int lane = threadIdx.x % LANES;
  PhiloxKey key{};
  if (drop) key = philox_key(p.mask);
  float ag[PARTS][E], ab[PARTS][E];
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) ag[k][e] = ab[k][e] = 0.f;
  uint64_t r = (uint64_t)blockIdx.x * PER + threadIdx.x / LANES;
#pragma unroll 1
  for (uint32_t t = 0; t < turns; ++t, r += (uint64_t)gridDim.x * PER) {
    const bool on = r < p.rows;
    const Row w = row_of(p, on ? (uint32_t)r : 0);
    Raw<S, VEC> rx[PARTS], rd[PARTS];
    Raw<IO, VEC> ry[PARTS];
    const int64_t ax = w.at(p.x1.s), ad = w.at(p.dx1.s), ay = w.at(p.dy.s);
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
      load_part<S, VEC>(rx[k], p.x1.p, ax, c, p.C, on);
      load_part<IO, VEC>(ry[k], p.dy.p, ay, c, p.C, on);
      if (p.dx1.p) load_part<S, VEC>(rd[k], p.dx1.p, ad, c, p.C, on);
    }
    float h[PARTS][E], g[PARTS][E];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      rx[k].get(h[k]);
      ry[k].get(g[k]);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += h[k][e];
    }
    float mean = 0.f;
    if (!p.rms) mean = row_sum<LANES>(sum, sums, 0) * p.inv_c;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = L::has(p.C, L::chan(lane, k), e) ? h[k][e] - mean : 0.f;
        h[k][e] = d;
        sq = fmaf(d, d, sq);
      }
    const float rstd = rsqrtf(row_sum<LANES>(sq, sums, 1) * p.inv_c + p.eps);
    float m1 = 0.f, m2 = 0.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = L::chan(lane, k) + L::off(e);
        h[k][e] *= rstd;
        ag[k][e] = fmaf(g[k][e], h[k][e], ag[k][e]);
        ab[k][e] += g[k][e];
        if (p.gamma && L::has(p.C, L::chan(lane, k), e)) g[k][e] *= p.gamma[c];
        m1 = fmaf(g[k][e], h[k][e], m1);
        m2 += g[k][e];
      }
    m1 = row_sum<LANES>(m1, sums, 2) * p.inv_c;
    m2 = p.rms ? 0.f : row_sum<LANES>(m2, sums, 3) * p.inv_c;
    const uint32_t mrow = drop ? (uint32_t)w.at(p.mask.s) : 0u;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const int c = L::chan(lane, k);
      float d[E];
      if (p.dx1.p) {
        rd[k].get(d);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = fmaf(rstd, fmaf(-h[k][e], m1, g[k][e]) - m2, d[e]);
      store_part<S, VEC>(p.dx.p, w.at(p.dx.s), c, p.C, on, d);
      if (p.du.p) {
        if (drop) {
          const uint32_t bits = keep_bits<VEC>(key, p.mask.threshold, c, mrow);
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] = (bits >> e & 1) ? d[e] * p.mask.scale : 0.f;
        }
        store_part<IO, VEC>(p.du.p, w.at(p.du.s), c, p.C, on, d);
      }
    }
    if constexpr (LANES > 32) __syncthreads();  // the next row's sums
  }
  // the row groups of the CTA, one after another
#pragma unroll 1
  for (int q = 0; q < PER; ++q) {
    if ((int)threadIdx.x / LANES == q)
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = L::chan(lane, k) + L::off(e);
          if (c < p.C) {
            part[c] = q ? part[c] + ag[k][e] : ag[k][e];
            part[p.C + c] = q ? part[p.C + c] + ab[k][e] : ab[k][e];
          }
        }
    __syncthreads();
  }
  float* out = p.ws + (int64_t)blockIdx.x * 2 * p.C;
  for (int c = threadIdx.x; c < 2 * p.C; c += kThreads) out[c] = part[c];
}

// Partial sums of `count` CTAs: 8 warps share 32 columns, each a stretch of the
// CTAs, joined in order.
template <typename T>
__global__ void __launch_bounds__(256) k_norm8_reduce(const Params p, int count) {
  __shared__ float buf[8][32];
  wait_for_earlier_work();
  let_next_start();
  const int warp = threadIdx.x >> 5, c = blockIdx.x * 32 + (threadIdx.x & 31);
  const int per = (count + 7) / 8, lo = warp * per, hi = min(count, lo + per);
  float s = 0.f;
  if (c < 2 * p.C)
#pragma unroll 8
    for (int k = lo; k < hi; ++k) s += p.ws[(int64_t)k * 2 * p.C + c];
  buf[warp][threadIdx.x & 31] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * p.C) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += buf[k][threadIdx.x];
    float* out = c < p.C ? p.dgamma : p.dbeta;
    if (out) out[c < p.C ? c : c - p.C] = s;
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

inline Params params_of(const Norm8Call& c) {
  Params p{};
  p.rows = (uint32_t)c.n[0] * (uint32_t)c.n[1] * (uint32_t)c.n[2];
  p.n1 = (uint32_t)c.n[1];
  p.n2 = (uint32_t)c.n[2];
  p.C = c.C;
  p.groups = (c.C + kGroup8 - 1) / kGroup8;
  p.inv_c = 1.0f / (float)c.C;
  p.eps = c.eps;
  p.rms = c.rms;
  p.mask = c.mask;
  p.x = c.x; p.u = c.u; p.x1 = c.x1;
  p.dx1 = c.dx1; p.dy = c.dy; p.dx = c.dx; p.du = c.du;
  p.codes = c.codes; p.scales = c.scales; p.scales_g = c.scales_g;
  for (int k = 0; k < 3; ++k) { p.codes_s[k] = c.codes_s[k]; p.scales_s[k] = c.scales_s[k]; }
  p.gamma = c.gamma; p.beta = c.beta;
  p.dgamma = c.dgamma; p.dbeta = c.dbeta; p.ws = c.ws;
  return p;
}

template <typename S, typename IO>
cudaError_t run_dropout(const Norm8Call& c, cudaStream_t st) {
  const Params p = params_of(c);
  const bool vec = c.C % 8 == 0 && aligned16(c.x, sizeof(S)) && aligned16(c.x1, sizeof(S)) &&
                   aligned16(c.u, sizeof(IO));
  const uint32_t per_row = vec ? (uint32_t)c.C / 8 : (uint32_t)p.groups;
  const uint64_t items = (uint64_t)p.rows * per_row, per_cta = vec ? 256 : 8;
  const uint64_t grid = (items + per_cta - 1) / per_cta;
  if (grid > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  return vec ? launch_early(k_dropout_add<S, IO, true>, (unsigned)grid, 256, 0, st, p, items, per_row, c.drop)
             : launch_early(k_dropout_add<S, IO, false>, (unsigned)grid, 256, 0, st, p, items, per_row, c.drop);
}

// The threads of a row and the parts of each, by the channel count: up to 32
// channels per thread, whole warps in one CTA beyond 1024 channels.
template <bool VEC, typename F>
cudaError_t by_width(int C, F&& f) {
#define EVO_N8(lanes, parts) return f(std::integral_constant<int, lanes>{}, std::integral_constant<int, parts>{})
  if constexpr (VEC) {
    if (C <= 64) EVO_N8(8, 1);
    if (C <= 128) EVO_N8(16, 1);
    if (C <= 256) EVO_N8(32, 1);
    if (C <= 512) EVO_N8(32, 2);
    if (C <= 1024) EVO_N8(32, 4);
    if (C <= 2048) EVO_N8(64, 4);
    EVO_N8(128, 4);
  } else {
    if (C <= 128) EVO_N8(32, 1);
    if (C <= 256) EVO_N8(32, 2);
    if (C <= 512) EVO_N8(32, 4);
    if (C <= 1024) EVO_N8(32, 8);
    if (C <= 2048) EVO_N8(64, 8);
    EVO_N8(128, 8);
  }
#undef EVO_N8
}

template <typename S, typename IO, bool VEC>
cudaError_t run_fwd_as(const Norm8Call& c, cudaStream_t st) {
  const Params p = params_of(c);
  return by_width<VEC>(c.C, [&](auto lanes, auto parts) {
    constexpr int L = decltype(lanes)::value, P = decltype(parts)::value;
    constexpr uint32_t per = kThreads / L;
    const int turns = 4;
    const uint32_t grid = (uint32_t)(((uint64_t)p.rows + per * turns - 1) / (per * turns));
    return launch_early(k_norm8_fwd<S, IO, L, P, VEC>, grid, kThreads, 0, st, p, turns, c.drop);
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
  const Params p = params_of(c);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return by_width<VEC>(c.C, [&](auto lanes, auto parts) {
    constexpr int L = decltype(lanes)::value, P = decltype(parts)::value;
    constexpr uint32_t per = kThreads / L;
    auto kern = k_norm8_bwd<S, IO, L, P, VEC>;
    const size_t smem = (size_t)2 * c.C * sizeof(float);
    int fit = 0;
    cudaError_t e2 = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, kThreads, smem);
    if (e2 != cudaSuccess) return e2;
    const uint32_t want = (uint32_t)(((uint64_t)p.rows + per - 1) / per);
    const uint32_t most = std::min<uint32_t>(kNorm8MaxCtas, (uint32_t)std::max(1, fit * sms));
    const uint32_t grid = std::min(want, most);
    const uint32_t turns = (want + grid - 1) / grid;
    e2 = launch_early(kern, grid, kThreads, smem, st, p, turns, c.drop);
    if (e2 != cudaSuccess || (!p.dgamma && !p.dbeta)) return e2;
    return launch_early(k_norm8_reduce<S>, (unsigned)(2 * c.C + 31) / 32, 256, 0, st, p, (int)grid);
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
