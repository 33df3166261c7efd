// A matrix in e4m3 with a power-of-two scale for each 128 elements of a row, of
// a column (stored transposed, so that a product over the rows reads it along
// memory), both from one read, or for each 128 x 128 block in both orders.
//
// Bound by memory: an element is read once and each copy written once.  A CTA
// takes a 128 x 128 tile, the largest piece that a scale spans in both
// directions; thread (ty, tx) holds the 8 x 8 elements of rows 8 ty and columns
// 8 tx in registers, so that the eight loads of 16 bytes are in flight at once,
// 16 neighbouring threads see a row and 16 strided ones a column, and eight
// codes of a column are one 8-byte unit of the transposed tile.  That goes
// through shared memory, where a unit's place in its 128-byte column is XORed
// with the column's tx: 16 threads of a warp then hit 16 different units.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.cuh"
#include "quantize8.h"
#include "scale8.cuh"

namespace evo {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Load;
template <>
struct Load<__nv_bfloat16> {
  static __device__ __forceinline__ void eight(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Load<float> {
  static __device__ __forceinline__ void eight(const float* p, float (&f)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};

__device__ __forceinline__ uint2 eight_codes(const float (&f)[8], float inv) {
  return make_uint2(e4m3_pair(f[0], f[1], inv) | e4m3_pair(f[2], f[3], inv) << 16,
                    e4m3_pair(f[4], f[5], inv) | e4m3_pair(f[6], f[7], inv) << 16);
}
// The first `n` (1 to 8) of eight codes.
__device__ __forceinline__ void put_codes(uint8_t* p, uint2 q, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = q;
    return;
  }
  const uint64_t v = (uint64_t)q.y << 32 | q.x;
  for (int e = 0; e < n; ++e) p[e] = (uint8_t)(v >> 8 * e);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_quantize8(const Quantize8Call c, uint32_t tiles_k) {
  __shared__ float col_max[8][kGroup8];
  __shared__ float col_inv[kGroup8];
  __shared__ __align__(16) uint8_t turned[kGroup8 * kGroup8];
  wait_for_earlier_work();
  let_next_start();
  const uint32_t tr = blockIdx.x / tiles_k, tk = blockIdx.x - tr * tiles_k;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t r0 = (int64_t)tr * kGroup8 + ty * 8;
  const int64_t k0 = (int64_t)tk * kGroup8 + tx * 8;
  const int nk = (int)min((int64_t)8, c.K - k0);  // this thread's columns (may be negative)
  const int nr = (int)min((int64_t)8, c.R - r0);  // and rows
  float f[8][8];
  const T* x = static_cast<const T*>(c.x);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (VEC && i < nr && nk > 0) {  // (K is a multiple of 8)
      Load<T>::eight(x + (r0 + i) * c.ld + k0, f[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = !VEC && i < nr && e < nk ? Load<T>::one(x + (r0 + i) * c.ld + k0 + e) : 0.f;
    }
  }
  const bool cols = c.codes_t != nullptr || c.blocks;
  float block = 0.f;
  if (cols) {
    // column maxima: 8 rows of this thread, the other half of the warp, 8 warps
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(f[i][e]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if ((threadIdx.x & 16) == 0) col_max[warp][tx * 8 + e] = m;
    }
    __syncthreads();
    if (threadIdx.x < kGroup8) {
      float m = col_max[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < 8; ++k) m = fmaxf(m, col_max[k][threadIdx.x]);
      if (!c.blocks) {
        const uint32_t code = scale_code(m);
        m = scale_inverse(code);
        const int64_t k = (int64_t)tk * kGroup8 + threadIdx.x;
        if (k < c.K) c.scales_t[k * c.st_row + (int64_t)tr * c.st_group] = (uint8_t)code;
      }
      col_inv[threadIdx.x] = m;
    }
    __syncthreads();
    if (c.blocks) {
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) m = fmaxf(m, col_inv[(threadIdx.x & 31) + 32 * k]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t code = scale_code(m);
      block = scale_inverse(code);
      if (threadIdx.x == 0) c.scales[(int64_t)tr * c.s_row + (int64_t)tk * c.s_group] = (uint8_t)code;
    }
  }
  if (c.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float inv = block;
      if (!c.blocks) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_abs(f[i][e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t code = scale_code(m);
        inv = scale_inverse(code);
        if (tx == 0 && i < nr) c.scales[(r0 + i) * c.s_row + (int64_t)tk * c.s_group] = (uint8_t)code;
      }
      if (i < nr && nk > 0) put_codes(c.codes + (r0 + i) * c.ldc + k0, eight_codes(f[i], inv), nk);
    }
  }
  if (c.codes_t) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = tx * 8 + e;
      const float inv = c.blocks ? block : col_inv[col];
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = f[i][e];
      *reinterpret_cast<uint2*>(turned + col * kGroup8 + ((ty ^ tx) << 3)) = eight_codes(t, inv);
    }
    __syncthreads();
    // eight threads write a column of the tile (128 bytes), 16 bytes each
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
      const int col = pass * 32 + (threadIdx.x >> 3), unit = (threadIdx.x & 7) * 2;
      const int64_t k = (int64_t)tk * kGroup8 + col, r = (int64_t)tr * kGroup8 + unit * 8;
      const uint2 a = *reinterpret_cast<const uint2*>(turned + col * kGroup8 + ((unit ^ (col >> 3)) << 3));
      const uint2 b = *reinterpret_cast<const uint2*>(turned + col * kGroup8 + (((unit + 1) ^ (col >> 3)) << 3));
      if (k >= c.K) continue;
      uint8_t* to = c.codes_t + k * c.ldt + r;
      if (r + 16 <= c.R) {
        *reinterpret_cast<uint4*>(to) = make_uint4(a.x, a.y, b.x, b.y);
      } else if (r < c.R) {
        put_codes(to, a, (int)min((int64_t)8, c.R - r));
        if (r + 8 < c.R) put_codes(to + 8, b, (int)min((int64_t)8, c.R - r - 8));
      }
    }
  }
}

template <typename T>
cudaError_t run(const Quantize8Call& c, cudaStream_t st) {
  const uint64_t tiles_k = (uint64_t)((c.K + kGroup8 - 1) / kGroup8);
  const uint64_t tiles = (uint64_t)((c.R + kGroup8 - 1) / kGroup8) * tiles_k;
  if (tiles > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  const bool vec = c.K % 8 == 0 && reinterpret_cast<uintptr_t>(c.x) % 16 == 0 &&
                   c.ld * (int64_t)sizeof(T) % 16 == 0;
  return vec ? launch_early(k_quantize8<T, true>, (unsigned)tiles, kThreads, 0, st, c, (uint32_t)tiles_k)
             : launch_early(k_quantize8<T, false>, (unsigned)tiles, kThreads, 0, st, c, (uint32_t)tiles_k);
}

}  // namespace

cudaError_t quantize8(const Quantize8Call& c, bool f32, cudaStream_t st) {
  return f32 ? run<float>(c, st) : run<__nv_bfloat16>(c, st);
}

}  // namespace evo
