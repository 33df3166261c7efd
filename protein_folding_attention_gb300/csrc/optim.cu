// One AdamW step over many tensors, and the norm of all their gradients.
//
//   g' = clip g    m = b1 m + (1 - b1) g'    v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by HBM: 28 bytes per element with fp32 states, bf16 gradients and a
// bf16 copy, 16 with 8-bit states, against about 20 fp32 operations.
//
// The tensors of a launch are a table in the kernel's parameters (up to 400
// rows of 72 bytes: no copy to the device, nothing to keep alive, and a
// captured launch carries its own table).  Each CTA takes an even share of the
// chunks of all tensors in order, so it looks its first tensor up once and
// walks on from there; small tensors cost a chunk each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "optim.h"

namespace evo {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = EVOATTN_ADAMW_BLOCK;  // elements per warp and turn; a block of the 8-bit states
constexpr int kStepChunk = kWarps * kBlock;  // elements per CTA and turn
constexpr int kNormUnroll = 4;
constexpr int kNormChunk = kNormUnroll * kThreads * 8;
constexpr int kNormCtas = 1216;              // partial sums per launch at most (8 per SM)
static_assert(kBlock == 256, "a lane holds 8 elements of a block");

struct Entry {
  float* p;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  __nv_bfloat16* copy;
  int64_t n;
  float wd;
  uint32_t flags;  // kGradBf16, kVec
};
constexpr uint32_t kGradBf16 = 1u, kVec = 2u;

constexpr int kMaxTensors = 400;
template <int T>
struct Table {
  Entry e[T];
  uint32_t start[T + 1];  // first chunk of each tensor
  int count;
};
template <int T>
struct StepParams {
  Table<T> t;
  evoattn_optim_state* state;
  const float* lr_device;
  float lr, b1, b1c, b2, b2c, log_b1, log_b2, eps;
  int clip, last;  // last: this launch counts the step up
};
template <int T>
struct NormParams {
  Table<T> t;
  evoattn_optim_state* state;
  double* part;    // this launch's partial sums; all launches' begin at part_all
  double* part_all;
  int parts_before, last;
  float max_norm;
};
static_assert(sizeof(StepParams<kMaxTensors>) <= 32764 && sizeof(NormParams<kMaxTensors>) <= 32764,
              "kernel parameters");

// The tensor that holds a chunk.
template <int T>
__device__ __forceinline__ int find_tensor(const Table<T>& t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.start[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// This CTA's even share [first, end) of the chunks.
template <int T>
__device__ __forceinline__ void my_share(const Table<T>& t, uint32_t* first, uint32_t* end) {
  const uint64_t total = t.start[t.count];
  *first = (uint32_t)(total * blockIdx.x / gridDim.x);
  *end = (uint32_t)(total * (blockIdx.x + 1) / gridDim.x);
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// e4m3 codes: four to a word, rounded to nearest even (beyond 448 to 448).
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ void from_e4m3(uint32_t w, float* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f16x2;
    const uint16_t two = (uint16_t)(w >> (16 * h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f16x2) : "h"(two));
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
        : "=f"(v[2 * h]), "=f"(v[2 * h + 1])
        : "r"(f16x2));
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Elements of a lane within its warp's block of 256: 4 * lane + {0..3} of each
// half, so that an access of the warp covers 128 elements without gaps.
__device__ __forceinline__ int element(int lane, int k) { return (k >> 2) * 128 + 4 * lane + (k & 3); }

template <bool BITS8, int T>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ StepParams<T> P) {
  // every CTA reads the step before the last one to do so counts it up
  const float t = (float)(P.state->step + 1);
  const float clip = P.clip ? P.state->clip : 1.f;
  const bool skip = P.clip && P.state->skip;
  const float lr = P.lr_device ? *P.lr_device : P.lr;
  if (P.last) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(&P.state->ticket[0], 1u) == gridDim.x - 1) {
        P.state->ticket[0] = 0;
        if (!skip) P.state->step += 1;
      }
    }
  }
  if (skip) return;
  // 1 - b^t without cancellation
  const float c1 = -expm1f(t * P.log_b1), c2 = -expm1f(t * P.log_b2);
  const float rate = lr / c1, root = rsqrtf(c2);

  uint32_t chunk, end;
  my_share(P.t, &chunk, &end);
  if (chunk >= end) return;
  int i = find_tensor(P.t, chunk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (; chunk < end; ++chunk) {
    while (chunk >= P.t.start[i + 1]) ++i;
    const Entry& e = P.t.e[i];
    const int64_t base = (int64_t)(chunk - P.t.start[i]) * kStepChunk + warp * kBlock;
    if (base >= e.n) continue;
    const bool vec = (e.flags & kVec) && base + kBlock <= e.n;
    float p[8], g[8], m[8], v[8];
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = base + element(lane, 4 * h);
        *reinterpret_cast<float4*>(p + 4 * h) = *reinterpret_cast<const float4*>(e.p + at);
        if (e.flags & kGradBf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(e.g) + at);
          g[4 * h] = bf_lo(w.x); g[4 * h + 1] = bf_hi(w.x);
          g[4 * h + 2] = bf_lo(w.y); g[4 * h + 3] = bf_hi(w.y);
        } else {
          *reinterpret_cast<float4*>(g + 4 * h) =
              *reinterpret_cast<const float4*>(static_cast<const float*>(e.g) + at);
        }
        if (BITS8) {
          from_e4m3(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.m) + at), m + 4 * h);
          from_e4m3(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.v) + at), v + 4 * h);
        } else {
          *reinterpret_cast<float4*>(m + 4 * h) =
              *reinterpret_cast<const float4*>(static_cast<const float*>(e.m) + at);
          *reinterpret_cast<float4*>(v + 4 * h) =
              *reinterpret_cast<const float4*>(static_cast<const float*>(e.v) + at);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t at = base + element(lane, k);
        const bool ok = at < e.n;
        p[k] = ok ? e.p[at] : 0.f;
        g[k] = !ok ? 0.f
                   : (e.flags & kGradBf16) ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.g)[at])
                                           : static_cast<const float*>(e.g)[at];
        if (BITS8) {
          float w[4];
          from_e4m3(ok ? static_cast<const uint8_t*>(e.m)[at] : 0u, w);
          m[k] = w[0];
          from_e4m3(ok ? static_cast<const uint8_t*>(e.v)[at] : 0u, w);
          v[k] = w[0];
        } else {
          m[k] = ok ? static_cast<const float*>(e.m)[at] : 0.f;
          v[k] = ok ? static_cast<const float*>(e.v)[at] : 0.f;
        }
      }
    }
    const float keep = 1.f - lr * e.wd;
    float ms = 0.f, vs = 0.f;
    if (BITS8) {
      ms = e.ms[base / kBlock];
      vs = e.vs[base / kBlock];
    }
    // one rounding per operation (no fused multiply-add), so that the codes of
    // the 8-bit states do not depend on how an expression is compiled
    float top_m = 0.f, top_v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gk = __fmul_rn(clip, g[k]);
      if (BITS8) {
        m[k] = __fmul_rn(m[k], ms);
        v[k] = __fmul_rn(v[k], vs);
        v[k] = __fmul_rn(v[k], v[k]);
      }
      m[k] = __fadd_rn(__fmul_rn(P.b1, m[k]), __fmul_rn(P.b1c, gk));
      v[k] = __fadd_rn(__fmul_rn(P.b2, v[k]), __fmul_rn(P.b2c, __fmul_rn(gk, gk)));
      const float r = BITS8 ? __fsqrt_rn(v[k]) : sqrtf(v[k]);
      p[k] = fmaf(-rate, __fdividef(m[k], fmaf(r, root, P.eps)), p[k] * keep);
      if (BITS8) {
        v[k] = r;  // the root is what is stored
        top_m = fmaxf(top_m, fabsf(m[k]));
        top_v = fmaxf(top_v, r);
      }
    }
    if (BITS8) {
      top_m = warp_max(top_m);
      top_v = warp_max(top_v);
      const bool hold_m = top_m >= 0x1p-100f, hold_v = top_v >= 0x1p-100f;
      const float im = hold_m ? __fdiv_rn(448.f, top_m) : 0.f;
      const float iv = hold_v ? __fdiv_rn(448.f, top_v) : 0.f;
      if (lane == 0) {
        e.ms[base / kBlock] = hold_m ? __fdiv_rn(top_m, 448.f) : 0.f;
        e.vs[base / kBlock] = hold_v ? __fdiv_rn(top_v, 448.f) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = __fmul_rn(m[k], im);
        // a positive root takes at least the smallest code (2^-9)
        const float q = __fmul_rn(v[k], iv);
        v[k] = v[k] > 0.f && hold_v ? fmaxf(q, 0x1p-9f) : q;
      }
    }
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = base + element(lane, 4 * h);
        const float* q = p + 4 * h;
        *reinterpret_cast<float4*>(e.p + at) = make_float4(q[0], q[1], q[2], q[3]);
        if (e.copy) {
          uint2 w;
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(q[1]), "f"(q[0]));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(q[3]), "f"(q[2]));
          *reinterpret_cast<uint2*>(e.copy + at) = w;
        }
        const float *mk = m + 4 * h, *vk = v + 4 * h;
        if (BITS8) {
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.m) + at) = to_e4m3(mk[0], mk[1], mk[2], mk[3]);
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.v) + at) = to_e4m3(vk[0], vk[1], vk[2], vk[3]);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(e.m) + at) = make_float4(mk[0], mk[1], mk[2], mk[3]);
          *reinterpret_cast<float4*>(static_cast<float*>(e.v) + at) = make_float4(vk[0], vk[1], vk[2], vk[3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t at = base + element(lane, k);
        if (at >= e.n) continue;
        e.p[at] = p[k];
        if (e.copy) e.copy[at] = __float2bfloat16_rn(p[k]);
        if (BITS8) {
          static_cast<uint8_t*>(e.m)[at] = (uint8_t)to_e4m3(m[k], 0.f, 0.f, 0.f);
          static_cast<uint8_t*>(e.v)[at] = (uint8_t)to_e4m3(v[k], 0.f, 0.f, 0.f);
        } else {
          static_cast<float*>(e.m)[at] = m[k];
          static_cast<float*>(e.v)[at] = v[k];
        }
      }
    }
  }
}

// Sum over a CTA in fp64, valid in thread 0.
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

// The last CTA to finish adds all partial sums in order, so the order of
// arrival changes nothing.
template <int T>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ NormParams<T> P) {
  uint32_t chunk, end;
  my_share(P.t, &chunk, &end);
  double total = 0.0;
  if (chunk < end) {
    int i = find_tensor(P.t, chunk);
    for (; chunk < end; ++chunk) {
      while (chunk >= P.t.start[i + 1]) ++i;
      const Entry& e = P.t.e[i];
      const int64_t base = (int64_t)(chunk - P.t.start[i]) * kNormChunk;
      const bool vec = (e.flags & kVec) && base + kNormChunk <= e.n;
      float s[kNormUnroll];
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) s[u] = 0.f;
      if (vec && (e.flags & kGradBf16)) {
        uint4 w[kNormUnroll];
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(e.g) + base + 8 * threadIdx.x;
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u)
          w[u] = *reinterpret_cast<const uint4*>(src + u * kThreads * 8);
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
          const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[u] = fmaf(bf_lo(q[k]), bf_lo(q[k]), s[u]);
            s[u] = fmaf(bf_hi(q[k]), bf_hi(q[k]), s[u]);
          }
        }
      } else if (vec) {
        float4 w[2 * kNormUnroll];
        const float* src = static_cast<const float*>(e.g) + base + 4 * threadIdx.x;
#pragma unroll
        for (int u = 0; u < 2 * kNormUnroll; ++u)
          w[u] = *reinterpret_cast<const float4*>(src + u * kThreads * 4);
#pragma unroll
        for (int u = 0; u < 2 * kNormUnroll; ++u) {
          float& d = s[u >> 1];
          d = fmaf(w[u].x, w[u].x, d);
          d = fmaf(w[u].y, w[u].y, d);
          d = fmaf(w[u].z, w[u].z, d);
          d = fmaf(w[u].w, w[u].w, d);
        }
      } else {
        const int64_t stop = min(e.n, base + (int64_t)kNormChunk);
#pragma unroll 4
        for (int64_t at = base + threadIdx.x; at < stop; at += kThreads) {
          const float g = (e.flags & kGradBf16)
                              ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.g)[at])
                              : static_cast<const float*>(e.g)[at];
          s[0] = fmaf(g, g, s[0]);
        }
      }
      total += (double)((s[0] + s[1]) + (s[2] + s[3]));
    }
  }
  total = cta_sum(total);
  __shared__ int is_last;
  if (threadIdx.x == 0) {
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
  __syncthreads();  // cta_sum's shared sums are reused
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

// Rows [from, from + count) of the call's tensors; false when the chunks do
// not fit 32 bits.
template <int T>
bool fill_table(Table<T>& t, const evoattn_adamw_tensor* src, int count, int chunk_elems, int bits) {
  uint64_t chunks = 0;
  t.count = 0;
  for (int i = 0; i < count; ++i) {
    const evoattn_adamw_tensor& s = src[i];
    if (s.n == 0) continue;
    Entry& e = t.e[t.count];
    e = Entry{s.param, s.grad, s.exp_avg, s.exp_avg_sq, s.exp_avg_scale, s.exp_avg_sq_scale,
              static_cast<__nv_bfloat16*>(s.copy), s.n, s.weight_decay, 0u};
    const bool bf16 = s.grad_dtype == EVOATTN_BF16;
    bool vec = aligned(s.grad, 16);
    if (bits) {
      const size_t state = bits == 8 ? 4 : 16;
      vec = vec && aligned(s.param, 16) && aligned(s.exp_avg, state) && aligned(s.exp_avg_sq, state) &&
            aligned(s.copy, 8);
    }
    e.flags = (bf16 ? kGradBf16 : 0u) | (vec ? kVec : 0u);
    t.start[t.count++] = (uint32_t)chunks;
    chunks += (uint64_t)(s.n + chunk_elems - 1) / (uint64_t)chunk_elems;
    if (chunks > 0x7FFFFFFFull) return false;
  }
  if (t.count == 0) {  // nothing to do but the bookkeeping
    t.start[0] = 0;
    t.count = 1;
    t.e[0] = Entry{};
  }
  t.start[t.count] = (uint32_t)chunks;
  return true;
}

// Resident CTAs of a kernel on the current device, looked up once.
template <typename K>
cudaError_t resident_ctas(K kernel, std::atomic<int> (&cache)[64], int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *n = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (*n > 0) return cudaSuccess;
  int sms = 0, per = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, 0);
  if (e != cudaSuccess) return e;
  *n = std::max(1, sms) * std::max(1, per);
  if (dev < 64) cache[dev].store(*n, std::memory_order_relaxed);
  return cudaSuccess;
}

template <bool BITS8, int T>
cudaError_t step_part(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                      evoattn_optim_state* state, bool last, cudaStream_t st) {
  static std::atomic<int> cache[64];
  StepParams<T> P;
  if (!fill_table(P.t, t, count, kStepChunk, BITS8 ? 8 : 32)) return cudaErrorInvalidConfiguration;
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
  P.clip = s.clip ? 1 : 0;
  P.last = last ? 1 : 0;
  int ctas = 0;
  cudaError_t e = resident_ctas(k_adamw<BITS8, T>, cache, &ctas);
  if (e != cudaSuccess) return e;
  const unsigned grid = std::max(1u, std::min<unsigned>(P.t.start[P.t.count], (unsigned)ctas));
  k_adamw<BITS8, T><<<grid, kThreads, 0, st>>>(P);
  return cudaGetLastError();
}

template <bool BITS8>
cudaError_t step_all(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                     evoattn_optim_state* state, cudaStream_t st) {
  for (int from = 0; from < count; from += kMaxTensors) {
    const int k = std::min(kMaxTensors, count - from);
    const bool last = from + k == count;
    // (a short table keeps a launch of few tensors short)
    const cudaError_t e = k <= 32 ? step_part<BITS8, 32>(t + from, k, s, state, last, st)
                                  : step_part<BITS8, kMaxTensors>(t + from, k, s, state, last, st);
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
  if (!fill_table(P.t, t, count, kNormChunk, 0)) return cudaErrorInvalidConfiguration;
  P.state = state;
  P.part_all = part_all;
  P.part = part_all + *parts;
  P.parts_before = *parts;
  P.last = last ? 1 : 0;
  P.max_norm = max_norm;
  int ctas = 0;
  cudaError_t e = resident_ctas(k_grad_norm<T>, cache, &ctas);
  if (e != cudaSuccess) return e;
  ctas = std::min(ctas, kNormCtas);
  const unsigned grid = std::max(1u, std::min<unsigned>(P.t.start[P.t.count], (unsigned)ctas));
  k_grad_norm<T><<<grid, kThreads, 0, st>>>(P);
  *parts += (int)grid;
  return cudaGetLastError();
}

}  // namespace

size_t grad_norm_workspace_bytes(int count) {
  return (size_t)((count + kMaxTensors - 1) / kMaxTensors) * kNormCtas * sizeof(double);
}

cudaError_t grad_norm(const evoattn_adamw_tensor* t, int count, float max_norm,
                      evoattn_optim_state* state, void* ws, cudaStream_t st) {
  int parts = 0;
  for (int from = 0; from < count; from += kMaxTensors) {
    const int k = std::min(kMaxTensors, count - from);
    const bool last = from + k == count;
    double* part = static_cast<double*>(ws);
    const cudaError_t e =
        k <= 32 ? norm_part<32>(t + from, k, max_norm, state, part, &parts, last, st)
                : norm_part<kMaxTensors>(t + from, k, max_norm, state, part, &parts, last, st);
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
