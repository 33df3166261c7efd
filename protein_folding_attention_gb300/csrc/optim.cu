// One AdamW step over many tensors, and the norm of all their gradients.
//
//   g' = clip g    m = b1 m + (1 - b1) g'    v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by HBM: 28 bytes per element with fp32 states, bf16 gradients and a
// bf16 copy, 16 with 8-bit states, against about 20 and 30 fp32 operations.
//
// The tensors of a launch are a table in the kernel's parameters (no copy to
// the device, nothing to keep alive, and a captured launch carries its own
// table).  All tensors are cut into blocks of 256 elements; small tensors cost
// a block each.  All warps of the launch sweep over the blocks together, a
// block each at a time: the memory then sees a few narrow fronts that move
// on, not a stream per CTA (107M parameters with 8-bit states: 355 us with a
// consecutive share of the blocks for each CTA, 264 us so).  Each warp copies
// its coming blocks into a ring in shared memory (cp.async): what is in flight
// does not depend on how many warps are between loading and storing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.cuh"
#include "optim.h"

namespace evo {
namespace {

constexpr int kThreads = 256;  // of a CTA of the norm's kernel
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = EVOATTN_ADAMW_BLOCK;  // elements a warp works on at a time
static_assert(kBlock == 256, "a lane holds 8 elements of a block");
constexpr int kCoarse = 1024;    // entries of the table from blocks to tensors
constexpr int kNormCtas = 912;   // partial sums of a norm's launch at most
constexpr int kNormUnroll = 4;   // blocks that a warp of the norm loads at once
constexpr int kNormUnit = kNormUnroll * kBlock;

// Flags of a tensor, above the 48 bits of its element count.
constexpr uint64_t kGradBf16 = 1ull << 48, kVec = 1ull << 49, kCount = (1ull << 48) - 1;

template <bool BITS8>
struct Entry {
  float* p;
  const void* g;
  void *m, *v;
  __nv_bfloat16* copy;
  uint64_t n;      // elements and flags
  float wd;
  uint32_t start;  // its first block
};
template <>
struct Entry<true> {
  float* p;
  const void* g;
  void *m, *v;
  __nv_bfloat16* copy;
  uint64_t n;
  float wd;
  uint32_t start;
  float *ms, *vs;
};

// Tensors of a launch: as many as the 32,764 bytes of kernel parameters hold,
// or few, which keeps the launch short.
template <bool BITS8>
constexpr int kManyTensors = BITS8 ? 416 : 536;
constexpr int kFewTensors = 32;

template <bool BITS8, int T>
struct StepParams {
  Entry<BITS8> e[T + 1];    // (the last one's successor holds the end)
  uint16_t coarse[kCoarse];  // the tensor that holds block k << shift
  int shift;
  evoattn_optim_state* state;
  const float* lr_device;
  float lr, b1, b1c, b2, b2c, log_b1, log_b2, eps;
  float one;       // 1, see sum2()
  int clip, last;  // last: this launch counts the step up
  uint32_t blocks;
};

struct NormEntry {
  const void* g;
  uint64_t n;
};
constexpr int kNormTensors = 1408;
template <int T>
struct NormParams {
  NormEntry e[T];
  uint32_t start[T + 1];
  uint16_t coarse[kCoarse];
  int shift;
  evoattn_optim_state* state;
  double* part;      // this launch's partial sums; all launches' begin at part_all
  double* part_all;
  int parts_before, last;
  float max_norm;
  uint32_t units;
};
static_assert(sizeof(StepParams<false, kManyTensors<false>>) <= 32764 &&
                  sizeof(StepParams<true, kManyTensors<true>>) <= 32764 &&
                  sizeof(NormParams<kNormTensors>) <= 32764,
              "kernel parameters");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// e4m3 codes: four to a word, rounded to nearest even (beyond 448 to 448).
__device__ __forceinline__ uint32_t to_e4m3(float2 a, float2 b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ void from_e4m3(uint32_t w, float2* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f16x2;
    const uint16_t two = (uint16_t)(w >> (16 * h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f16x2) : "h"(two));
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
        : "=f"(v[h].x), "=f"(v[h].y)
        : "r"(f16x2));
  }
}
__device__ __forceinline__ float sqrt_approx(float a) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float a) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float rcp_approx(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
// 448 (1 / top), 0 for a block that is held as zeros.
constexpr float kLeast = 0x1p-100f;
__device__ __forceinline__ float inverse448(float top) {
  return top >= kLeast ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// a + b, where a or b may be a product that has to be rounded before.  As a
// fused operation with a factor that is not known when the kernel is compiled:
// mul2 and add2 one after the other give the bits of one fma2 (a fifth of the
// scales was off by an ulp).  `one` is 1 and comes in as a parameter of the kernel.
__device__ __forceinline__ float2 sum2(float2 a, float2 b, float one) { return fma2(a, both(one), b); }

// Square roots, rounded to nearest, of a lane's eight values.  Inside the range
// where no step overflows or loses bits: from a = v y, y near 1 / sqrt(v), one
// Newton step a + (v - a^2) y / 2 with the residual exact in fp32 (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34, 1990).  It gave the correctly rounded root for every
// fp32 value in that range (all 1.6e9 compared on a GB300), so a root does not
// depend on which way the lane's other values take.  __fsqrt_rn for each of the
// eight: 271 us a step of 107M parameters, 258 so.
__device__ __forceinline__ void roots(const float2* v, float2* r) {
  const float low = fminf(fminf(fminf(v[0].x, v[0].y), fminf(v[1].x, v[1].y)),
                          fminf(fminf(v[2].x, v[2].y), fminf(v[3].x, v[3].y)));
  const float high = fmax3(fmax3(v[0].x, v[0].y, v[1].x), fmax3(v[1].y, v[2].x, v[2].y), fmaxf(v[3].x, v[3].y));
  if (low >= 0x1p-96f && high < 0x1p96f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 y = make_float2(rsqrt_approx(v[k].x), rsqrt_approx(v[k].y));
      const float2 a = mul2(v[k], y);
      const float2 rest = fma2(make_float2(-a.x, -a.y), a, v[k]);
      r[k] = fma2(rest, mul2(y, both(0.5f)), a);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = make_float2(__fsqrt_rn(v[k].x), __fsqrt_rn(v[k].y));
  }
}

__device__ __forceinline__ float2 warp_max(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
    v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
  }
  return v;
}

// A lane's 8 elements of a block are 4 * lane + {0..3} of each half, so that a
// warp's access covers 128 elements without gaps.
__device__ __forceinline__ int element(int lane, int k) { return (k >> 2) * 128 + 4 * lane + (k & 3); }

// A warp's stage of the ring: p, g (bf16 in the first half), then m and v,
// and with 8 bits their scales.
template <bool BITS8>
struct Ring {
  static constexpr uint32_t G = 1024, M = 2048, V = M + (BITS8 ? 256 : 1024);
  static constexpr uint32_t S = 2560;
  static_assert(!BITS8 || S + 8 <= 2576, "the scales are a stage's last");
  static constexpr uint32_t STAGE = BITS8 ? 2576 : 4096;
  static constexpr int STAGES = 3;
  static constexpr uint32_t BYTES = STAGE * STAGES;  // per warp
};

// Where a warp is: a block, the tensor that holds it, and that tensor's
// addresses as the lane uses them (looked up when a tensor begins).
template <bool BITS8, int T>
struct Cursor {
  uint32_t b, start, next;  // block; first block of this tensor and of the next
  uint32_t full;            // blocks of it that can be copied whole
  int i;
  bool bf16;
  const char *p, *g, *m, *v, *s;

  __device__ __forceinline__ void open(const StepParams<BITS8, T>& P, int lane) {
    i = P.coarse[b >> P.shift];
    while (b >= P.e[i + 1].start) ++i;
    const Entry<BITS8>& e = P.e[i];
    start = e.start;
    next = P.e[i + 1].start;
    full = e.n & kVec ? (uint32_t)((e.n & kCount) / kBlock) : 0u;
    bf16 = (e.n & kGradBf16) != 0;
    p = reinterpret_cast<const char*>(e.p) + lane * 16;
    g = static_cast<const char*>(e.g) + lane * 16;
    if constexpr (BITS8) {  // half a warp's copies each; two lanes copy the scales
      m = static_cast<const char*>(lane < 16 ? e.m : e.v) + (lane & 15) * 16;
      s = reinterpret_cast<const char*>(lane == 0 ? e.ms : e.vs);
    } else {
      m = static_cast<const char*>(e.m) + lane * 16;
      v = static_cast<const char*>(e.v) + lane * 16;
    }
  }
};

// WARPS: 8, with two CTAs per SM for 32-bit states and three for 8-bit ones
// (12M parameters of small tensors: 47.6 us with two, 45.3 with three); or, with
// 8-bit states, kFront in one CTA, which meet every fourth turn.  Left to
// themselves the warps drift apart over a long tensor and the front that they
// sweep widens (us of tensors of 62,000, 139,000, 0.4M and 18M elements on
// average: 118, 131, 126 and 306 apart, 121, 124, 113 and 258 so); with 32-bit
// states the two differ by less than 1 %.  More warps than 20 add nothing.
constexpr int kFront = 20;
template <bool BITS8, int T, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == kFront ? 1 : BITS8 ? 3 : 2)
    k_adamw(const __grid_constant__ StepParams<BITS8, T> P) {
  using R = Ring<BITS8>;
  extern __shared__ __align__(16) char smem[];
  wait_for_earlier_work();
  let_next_start();
  const float t = (float)(P.state->step + 1);
  const float clip = P.clip ? P.state->clip : 1.f;
  const bool skip = P.clip && P.state->skip;
  const float lr = P.lr_device ? *P.lr_device : P.lr;
  // Every CTA has read the step before the last one to end counts it up.
  __syncthreads();
  auto count_up = [&]() {
    if (!P.last || threadIdx.x != 0) return;
    __threadfence();
    if (atomicAdd(&P.state->ticket[0], 1u) == gridDim.x - 1) {
      P.state->ticket[0] = 0;
      if (!skip) P.state->step += 1;
    }
  };
  if (skip) {
    count_up();
    return;
  }
  // 1 - b^t without cancellation
  const float c1 = -expm1f(t * P.log_b1), c2 = -expm1f(t * P.log_b2);
  const float rate = lr / c1, root = rsqrtf(c2);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t end = P.blocks, hop = gridDim.x * WARPS;
  Cursor<BITS8, T> at;
  at.b = blockIdx.x * WARPS + warp;
  // turns that every warp of the launch takes
  uint32_t common = WARPS == kFront ? end / hop : 0;
  if (at.b >= end) {
    count_up();
    return;
  }
  at.open(P, lane);
  char* const ring = smem + warp * (R::STAGE * R::STAGES);
  const uint32_t ring_s = smem_u32(ring);

  auto fetch = [&](int stage, Cursor<BITS8, T>& c) {
    if (c.b < end) {
      if (c.b >= c.next) c.open(P, lane);
      const uint32_t rel = c.b - c.start;
      if (rel < c.full) {
        const uint32_t to = ring_s + stage * R::STAGE + lane * 16;
        const char* p = c.p + (uint64_t)rel * (kBlock * 4);
        copy16(to, p);
        copy16(to + 512, p + 512);
        const char* g = c.g + (uint64_t)rel * (c.bf16 ? kBlock * 2 : kBlock * 4);
        copy16(to + R::G, g);
        if (!c.bf16) copy16(to + R::G + 512, g + 512);
        if constexpr (BITS8) {
          copy16(to + R::M, c.m + (uint64_t)rel * kBlock);  // (V follows M by 256 bytes)
          if (lane < 2) copy4(ring_s + stage * R::STAGE + R::S + 4 * lane, c.s + (uint64_t)rel * 4);
        } else {
          const char *m = c.m + (uint64_t)rel * (kBlock * 4), *v = c.v + (uint64_t)rel * (kBlock * 4);
          copy16(to + R::M, m);
          copy16(to + R::M + 512, m + 512);
          copy16(to + R::V, v);
          copy16(to + R::V + 512, v + 512);
        }
      }
      c.b += hop;
    }
    copies_close();
  };

  Cursor<BITS8, T> ahead = at;
#pragma unroll
  for (int s = 0; s < R::STAGES - 1; ++s) fetch(s, ahead);
  int stage = 0;
  for (; at.b < end; at.b += hop) {
    if (at.b >= at.next) at.open(P, lane);
    const Entry<BITS8>& e = P.e[at.i];
    const uint32_t rel = at.b - at.start;
    const bool vec = rel < at.full;
    const int64_t base = (int64_t)rel * kBlock;
    if (WARPS == kFront && common > 0 && (--common & 3) == 0) __syncthreads();
    __syncwarp();  // the warp has read the stage that is filled next
    fetch(stage == 0 ? R::STAGES - 1 : stage - 1, ahead);
    copies_wait<R::STAGES - 1>();
    __syncwarp();
    const char* from = ring + stage * R::STAGE;
    stage = stage + 1 == R::STAGES ? 0 : stage + 1;

    float2 p[4], g[4], m[4], v[4];
    float ms = 0.f, vs = 0.f;
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        auto four = [&](uint32_t off, float2* d) {
          const float4 q = *reinterpret_cast<const float4*>(from + off + h * 512 + lane * 16);
          d[2 * h] = make_float2(q.x, q.y);
          d[2 * h + 1] = make_float2(q.z, q.w);
        };
        four(0, p);
        if (at.bf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(from + R::G + h * 256 + lane * 8);
          g[2 * h] = make_float2(bf16lo(w.x), bf16hi(w.x));
          g[2 * h + 1] = make_float2(bf16lo(w.y), bf16hi(w.y));
        } else {
          four(R::G, g);
        }
        if constexpr (BITS8) {
          from_e4m3(*reinterpret_cast<const uint32_t*>(from + R::M + h * 128 + lane * 4), m + 2 * h);
          from_e4m3(*reinterpret_cast<const uint32_t*>(from + R::V + h * 128 + lane * 4), v + 2 * h);
        } else {
          four(R::M, m);
          four(R::V, v);
        }
      }
      if constexpr (BITS8) {
        ms = *reinterpret_cast<const float*>(from + R::S);
        vs = *reinterpret_cast<const float*>(from + R::S + 4);
      }
    } else {
      const int64_t n = (int64_t)(e.n & kCount);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t a = base + element(lane, k);
        const bool ok = a < n;
        auto put = [&](float2* d, float x) { (k & 1 ? d[k >> 1].y : d[k >> 1].x) = x; };
        put(p, ok ? e.p[a] : 0.f);
        put(g, !ok ? 0.f
                   : at.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.g)[a])
                             : static_cast<const float*>(e.g)[a]);
        if constexpr (BITS8) {
          float2 w[2];
          from_e4m3(ok ? static_cast<const uint8_t*>(e.m)[a] : 0u, w);
          put(m, w[0].x);
          from_e4m3(ok ? static_cast<const uint8_t*>(e.v)[a] : 0u, w);
          put(v, w[0].x);
        } else {
          put(m, ok ? static_cast<const float*>(e.m)[a] : 0.f);
          put(v, ok ? static_cast<const float*>(e.v)[a] : 0.f);
        }
      }
      if constexpr (BITS8) {
        ms = e.ms[rel];
        vs = e.vs[rel];
      }
    }

    // With 8-bit states every operation is rounded by itself: a code then
    // depends on the formula alone, and the same operations elsewhere give the
    // same codes.
    const float keep = 1.f - lr * e.wd;
    float2 r[4], top = both(0.f);
    if constexpr (BITS8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 c = mul2(g[k], both(clip));
        m[k] = sum2(mul2(mul2(m[k], both(ms)), both(P.b1)), mul2(c, both(P.b1c)), P.one);
        v[k] = mul2(v[k], both(vs));
        v[k] = sum2(mul2(mul2(v[k], v[k]), both(P.b2)), mul2(mul2(c, c), both(P.b2c)), P.one);
      }
      roots(v, r);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 c = mul2(g[k], both(clip));
        m[k] = fma2(m[k], both(P.b1), mul2(c, both(P.b1c)));
        v[k] = fma2(v[k], both(P.b2), mul2(mul2(c, c), both(P.b2c)));
        r[k] = make_float2(sqrt_approx(v[k].x), sqrt_approx(v[k].y));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 d = fma2(r[k], both(root), both(P.eps));
      const float2 q = mul2(m[k], make_float2(rcp_approx(d.x), rcp_approx(d.y)));
      p[k] = fma2(q, both(-rate), mul2(p[k], both(keep)));
      if constexpr (BITS8) {
        top.x = fmax3(top.x, fabsf(m[k].x), fabsf(m[k].y));
        top.y = fmax3(top.y, r[k].x, r[k].y);
      }
    }
    if constexpr (BITS8) {
      top = warp_max(top);
      const float im = inverse448(top.x), iv = inverse448(top.y);
      if (lane < 2) {
        const float high = lane == 0 ? top.x : top.y;
        float* to = (lane == 0 ? e.ms : e.vs) + rel;
        *to = high >= kLeast ? __fmul_rn(high, 1.f / 448.f) : 0.f;
      }
      // a positive root takes at least the smallest code (2^-9)
      const float least = iv > 0.f ? 0x1p-9f : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = mul2(m[k], both(im));
        r[k] = mul2(r[k], both(iv));
        if (v[k].x > 0.f) r[k].x = fmaxf(r[k].x, least);
        if (v[k].y > 0.f) r[k].y = fmaxf(r[k].y, least);
      }
    }
    if (vec) {
      const int first = 4 * lane;
      float* to_p = e.p + base + first;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x = p[2 * h], y = p[2 * h + 1];
        *reinterpret_cast<float4*>(to_p + 128 * h) = make_float4(x.x, x.y, y.x, y.y);
      }
      if (e.copy) {
        __nv_bfloat16* to = e.copy + base + first;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 x = p[2 * h], y = p[2 * h + 1];
          *reinterpret_cast<uint2*>(to + 128 * h) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(y.x, y.y));
        }
      }
      if constexpr (BITS8) {
        uint8_t *to_m = static_cast<uint8_t*>(e.m) + base + first, *to_v = static_cast<uint8_t*>(e.v) + base + first;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          *reinterpret_cast<uint32_t*>(to_m + 128 * h) = to_e4m3(m[2 * h], m[2 * h + 1]);
          *reinterpret_cast<uint32_t*>(to_v + 128 * h) = to_e4m3(r[2 * h], r[2 * h + 1]);
        }
      } else {
        float *to_m = static_cast<float*>(e.m) + base + first, *to_v = static_cast<float*>(e.v) + base + first;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          *reinterpret_cast<float4*>(to_m + 128 * h) =
              make_float4(m[2 * h].x, m[2 * h].y, m[2 * h + 1].x, m[2 * h + 1].y);
          *reinterpret_cast<float4*>(to_v + 128 * h) =
              make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
        }
      }
    } else {
      const int64_t n = (int64_t)(e.n & kCount);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t a = base + element(lane, k);
        if (a >= n) continue;
        auto one = [&](const float2* d) { return k & 1 ? d[k >> 1].y : d[k >> 1].x; };
        e.p[a] = one(p);
        if (e.copy) e.copy[a] = __float2bfloat16_rn(one(p));
        if constexpr (BITS8) {
          static_cast<uint8_t*>(e.m)[a] = (uint8_t)to_e4m3(make_float2(one(m), 0.f), both(0.f));
          static_cast<uint8_t*>(e.v)[a] = (uint8_t)to_e4m3(make_float2(one(r), 0.f), both(0.f));
        } else {
          static_cast<float*>(e.m)[a] = one(m);
          static_cast<float*>(e.v)[a] = one(v);
        }
      }
    }
  }
  copies_wait<0>();
  count_up();
}

// Sum over a CTA, valid in thread 0.  (fp64 arithmetic is slow on this part,
// so only few fp64 additions are made.)
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double part[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < kWarps; ++i) v += part[i];
  return v;
}

// The launch's warps sweep over units of four blocks.  A block's squares are summed in fp32 (8 per lane),
// the blocks' sums with their rounding errors carried along.  The last CTA to
// finish adds all partial sums in order, so the order of arrival changes
// nothing.
template <int T>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ NormParams<T> P) {
  wait_for_earlier_work();
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float sum = 0.f, low = 0.f;
  for (uint32_t b = blockIdx.x * kWarps + warp; b < P.units; b += gridDim.x * kWarps) {
    int i = P.coarse[b >> P.shift];
    while (b >= P.start[i + 1]) ++i;
    const NormEntry& e = P.e[i];
    const int64_t base = (int64_t)(b - P.start[i]) * kNormUnit;
    // whole blocks of this unit, and elements behind them
    const int64_t left = (int64_t)(e.n & kCount) - base;
    const int count = left < kNormUnit ? (int)left : kNormUnit;
    const int whole = e.n & kVec ? count / kBlock : 0;
    float part[kNormUnroll];
    if (e.n & kGradBf16) {
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(e.g) + base;
      uint4 w[kNormUnroll];
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u)
        w[u] = u < whole ? *reinterpret_cast<const uint4*>(g + u * kBlock + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) {
        const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float2 t = both(0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = make_float2(bf16lo(q[k]), bf16hi(q[k]));
          t = fma2(x, x, t);
        }
        part[u] = t.x + t.y;
      }
      for (int k = whole * kBlock + lane; k < count; k += 32) {
        const float x = __bfloat162float(g[k]);
        part[0] = fmaf(x, x, part[0]);
      }
    } else {
      const float* g = static_cast<const float*>(e.g) + base;
      float4 w[kNormUnroll][2];
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[u][h] = u < whole ? *reinterpret_cast<const float4*>(g + u * kBlock + 128 * h + 4 * lane)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) {
        float2 t = both(0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 x = make_float2(w[u][h].x, w[u][h].y), y = make_float2(w[u][h].z, w[u][h].w);
          t = fma2(x, x, fma2(y, y, t));
        }
        part[u] = t.x + t.y;
      }
      for (int k = whole * kBlock + lane; k < count; k += 32) part[0] = fmaf(g[k], g[k], part[0]);
    }
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
      const float s = part[u];
      // sum + s exactly, as a rounded sum and its error (Knuth's two-sum)
      const float t = sum + s, back = t - sum;
      low += (sum - (t - back)) + (s - back);
      sum = t;
    }
  }
  // (an infinite sum's error would be NaN: the norm is infinite either way)
  float mine = isfinite(sum) ? sum + low : sum;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  __shared__ float sums[kWarps];
  __shared__ int is_last;
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int k = 0; k < kWarps; ++k) total += (double)sums[k];
    P.part[blockIdx.x] = total;
    __threadfence();
    is_last = P.last && atomicAdd(&P.state->ticket[1], 1u) == gridDim.x - 1;
  }
  if (!P.last) return;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  const int parts = P.parts_before + (int)gridDim.x;
  double all = 0.0;
  for (int k = threadIdx.x; k < parts; k += kThreads) all += __ldcg(P.part_all + k);
  all = cta_sum(all);
  if (threadIdx.x == 0) {
    const float norm = (float)sqrt(all);
    const bool bad = !isfinite(norm);
    P.state->norm = norm;
    P.state->clip = bad ? 0.f : fminf(1.f, P.max_norm / (norm + 1e-6f));
    P.state->skip = bad ? 1u : 0u;
    P.state->ticket[1] = 0;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

uint64_t grad_flags(const evoattn_adamw_tensor& s) {
  return (uint64_t)s.n | (s.grad_dtype == EVOATTN_BF16 ? kGradBf16 : 0) | (aligned(s.grad, 16) ? kVec : 0);
}

// Resident CTAs of a kernel on the current device, looked up once.
template <typename K>
cudaError_t resident_ctas(K kernel, int threads, size_t smem, std::atomic<int> (&cache)[64], int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *n = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (*n > 0) return cudaSuccess;
  int sms = 0, per = 0;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *n = std::max(1, sms) * std::max(1, per);
  if (dev < 64) cache[dev].store(*n, std::memory_order_relaxed);
  return cudaSuccess;
}

// The tensor that holds every 2^shift-th of `total` pieces.
template <typename StartOf>
int coarse_table(uint16_t (&table)[kCoarse], uint64_t total, StartOf start_of) {
  int shift = 0;
  while (total >> shift >= (uint64_t)kCoarse) ++shift;
  for (uint64_t c = 0, i = 0; (c << shift) < total; ++c) {
    while (c << shift >= start_of((int)i + 1)) ++i;
    table[c] = (uint16_t)i;
  }
  return shift;
}

template <bool BITS8, int T, int WARPS>
cudaError_t launch_step(const StepParams<BITS8, T>& P, cudaStream_t st) {
  static std::atomic<int> cache[64];
  constexpr size_t smem = (size_t)Ring<BITS8>::BYTES * WARPS;
  int ctas = 0;
  const cudaError_t e = resident_ctas(k_adamw<BITS8, T, WARPS>, WARPS * 32, smem, cache, &ctas);
  if (e != cudaSuccess) return e;
  // a warp for every block, at least one CTA for the bookkeeping
  const uint32_t want = std::max(1u, (P.blocks + WARPS - 1) / WARPS);
  return launch_early(k_adamw<BITS8, T, WARPS>, std::min(want, (uint32_t)ctas), WARPS * 32, smem, st, P);
}

template <bool BITS8, int T>
cudaError_t step_part(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                      evoattn_optim_state* state, bool last, cudaStream_t st) {
  StepParams<BITS8, T> P;
  uint64_t blocks = 0;
  int k = 0;
  for (int i = 0; i < count; ++i) {
    const evoattn_adamw_tensor& a = t[i];
    if (a.n == 0) continue;
    Entry<BITS8>& e = P.e[k++];
    e.p = a.param;
    e.g = a.grad;
    e.m = a.exp_avg;
    e.v = a.exp_avg_sq;
    e.copy = static_cast<__nv_bfloat16*>(a.copy);
    e.wd = a.weight_decay;
    e.n = grad_flags(a);
    if (!aligned(a.param, 16) || !aligned(a.exp_avg, 16) || !aligned(a.exp_avg_sq, 16) || !aligned(a.copy, 8))
      e.n &= ~kVec;
    if constexpr (BITS8) {
      e.ms = a.exp_avg_scale;
      e.vs = a.exp_avg_sq_scale;
    }
    e.start = (uint32_t)blocks;
    blocks += (uint64_t)(a.n + kBlock - 1) / kBlock;
    if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  }
  P.e[k].start = (uint32_t)blocks;
  P.blocks = (uint32_t)blocks;
  P.state = state;
  P.lr_device = s.lr_device;
  P.lr = s.lr;
  P.b1 = (float)s.beta1;
  P.b1c = (float)(1.0 - s.beta1);
  P.b2 = (float)s.beta2;
  P.b2c = (float)(1.0 - s.beta2);
  P.log_b1 = (float)log(s.beta1);
  P.log_b2 = (float)log(s.beta2);
  P.eps = s.eps;
  P.one = 1.f;
  P.clip = s.clip ? 1 : 0;
  P.last = last ? 1 : 0;
  P.shift = coarse_table(P.coarse, blocks, [&](int i) { return (uint64_t)P.e[i].start; });
  // large tensors: 512 blocks on average
  if constexpr (BITS8) {
    if (blocks >= 512ull * (uint64_t)std::max(k, 1)) return launch_step<BITS8, T, kFront>(P, st);
  }
  return launch_step<BITS8, T, 8>(P, st);
}

template <bool BITS8>
cudaError_t step_all(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                     evoattn_optim_state* state, cudaStream_t st) {
  constexpr int kMany = kManyTensors<BITS8>;
  for (int from = 0; from < count; from += kMany) {
    const int k = std::min(kMany, count - from);
    const bool last = from + k == count;
    const cudaError_t e = k <= kFewTensors ? step_part<BITS8, kFewTensors>(t + from, k, s, state, last, st)
                                           : step_part<BITS8, kMany>(t + from, k, s, state, last, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int T>
cudaError_t norm_part(const evoattn_adamw_tensor* t, int count, float max_norm,
                      evoattn_optim_state* state, double* part_all, int* parts, bool last,
                      cudaStream_t st) {
  static std::atomic<int> cache[64];
  NormParams<T> P;
  uint64_t units = 0;
  int k = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    P.e[k] = NormEntry{t[i].grad, grad_flags(t[i])};
    P.start[k++] = (uint32_t)units;
    units += (uint64_t)(t[i].n + kNormUnit - 1) / kNormUnit;
    if (units > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  }
  P.start[k] = (uint32_t)units;
  P.units = (uint32_t)units;
  P.state = state;
  P.part_all = part_all;
  P.part = part_all + *parts;
  P.parts_before = *parts;
  P.last = last ? 1 : 0;
  P.max_norm = max_norm;
  int ctas = 0;
  cudaError_t e = resident_ctas(k_grad_norm<T>, kThreads, 0, cache, &ctas);
  if (e != cudaSuccess) return e;
  // a CTA for every 8 units (one per warp), at least one for the bookkeeping
  const uint64_t want = std::max<uint64_t>(1, (units + kWarps - 1) / kWarps);
  const unsigned grid = (unsigned)std::min<uint64_t>(want, (uint64_t)std::min(ctas, kNormCtas));
  P.shift = coarse_table(P.coarse, units, [&](int i) { return (uint64_t)P.start[i]; });
  *parts += (int)grid;
  return launch_early(k_grad_norm<T>, grid, kThreads, 0, st, P);
}

}  // namespace

size_t grad_norm_workspace_bytes(int count) {
  return (size_t)((count + kNormTensors - 1) / kNormTensors) * kNormCtas * sizeof(double);
}

cudaError_t grad_norm(const evoattn_adamw_tensor* t, int count, float max_norm,
                      evoattn_optim_state* state, void* ws, cudaStream_t st) {
  int parts = 0;
  for (int from = 0; from < count; from += kNormTensors) {
    const int k = std::min(kNormTensors, count - from);
    const bool last = from + k == count;
    double* part = static_cast<double*>(ws);
    const cudaError_t e =
        k <= kFewTensors ? norm_part<kFewTensors>(t + from, k, max_norm, state, part, &parts, last, st)
                         : norm_part<kNormTensors>(t + from, k, max_norm, state, part, &parts, last, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t adamw32(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                    evoattn_optim_state* state, cudaStream_t st) {
  return step_all<false>(t, count, s, state, st);
}
cudaError_t adamw8(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                   evoattn_optim_state* state, cudaStream_t st) {
  return step_all<true>(t, count, s, state, st);
}

}  // namespace evo
