// A matrix in e4m3 with a power-of-two scale for each 128 elements of a row, of
// a column (stored transposed, so that a product over the rows reads it along
// memory), both from one read, or for each 128 x 128 block in both orders.
//
// Bound by memory: an element is read once and each copy written once.  A CTA
// takes a 128 x 128 tile, the largest piece that a scale spans in both
// directions; thread (ty, tx) of its 512 holds the 4 x 8 elements of rows 4 ty and
// columns 8 tx in registers, so that 16 neighbouring threads see a row and 32
// strided ones a column, four loads of 16 bytes per thread are in flight at once
// and four codes of a column are one word of the transposed tile.  That goes
// through shared memory, where a word's place in its 128-byte column is XORed with
// 2 tx: a warp's 32 words then hit 32 banks.
//
// With 4.4 bytes for each element (bf16, both copies) the memory rate leaves some
// 20 instructions per element: maxima are taken three operands at a time on
// magnitudes, which skips NaN, and infinities are looked for once per tile and
// turned into NaN, instead of a test per element.
//
// bf16 tiles come through a ring of two in shared memory, filled by cp.async by
// persistent CTAs while the tile before is worked on (a thread copies and reads
// only its own units: no barrier): with loads into registers 48 % of the warps that
// an SM can hold waited for them most of the time (102 us for 147,456 x 512 where
// the bytes take 45; with the ring, and without bank conflicts, 61; rows alone 67 ->
// 36 where they take 33).  fp32 tiles, twice the size, are loaded into registers.
// Rows that are no whole 16-byte units come through shared memory too: a warp
// reads a row's elements 32 at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "divide.cuh"
#include "launch.cuh"
#include "quantize8.h"
#include "scale8.cuh"

namespace evo {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 4;  // of a thread

template <typename T>
struct Load;
template <>
struct Load<__nv_bfloat16> {
  static constexpr int PITCH = 136;  // elements of a row in shared memory
  static __device__ __forceinline__ void unpack(const uint4& a, float (&f)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void eight(const __nv_bfloat16* p, float (&f)[8]) {
    unpack(__ldcs(reinterpret_cast<const uint4*>(p)), f);
  }
  static __device__ __forceinline__ void eight_shared(const __nv_bfloat16* p, float (&f)[8]) {
    unpack(*reinterpret_cast<const uint4*>(p), f);
  }
};
template <>
struct Load<float> {
  static constexpr int PITCH = 132;
  static __device__ __forceinline__ void unpack(const float4& a, const float4& b, float (&f)[8]) {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void eight(const float* p, float (&f)[8]) {
    unpack(__ldcs(reinterpret_cast<const float4*>(p)), __ldcs(reinterpret_cast<const float4*>(p) + 1), f);
  }
  static __device__ __forceinline__ void eight_shared(const float* p, float (&f)[8]) {
    unpack(reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1], f);
  }
};

// The first `n` (1 to 8) of eight codes.
__device__ __forceinline__ void put_codes(uint8_t* p, uint2 q, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = q;
    return;
  }
  const uint64_t v = (uint64_t)q.y << 32 | q.x;
  for (int e = 0; e < n; ++e) p[e] = (uint8_t)(v >> 8 * e);
}

// Shared memory of a CTA: the ring or the tile as it was read, and the transposed
// codes (which take the place of the latter).
template <typename T, bool VEC, bool COLS>
struct Smem {
  static constexpr bool RING = VEC && sizeof(T) == 2;
  static constexpr int DEPTH = 2;
  static constexpr uint32_t STAGE = kRows * kThreads * 16;
  static constexpr uint32_t RAW = VEC ? 0 : kGroup8 * Load<T>::PITCH * sizeof(T);
  static constexpr uint32_t TURNED = COLS ? kGroup8 * kGroup8 : 0;
  static constexpr uint32_t BYTES = RING ? DEPTH * STAGE + TURNED : RAW > TURNED ? RAW : TURNED;
};

template <typename T, bool VEC, bool COLS>
__global__ void __launch_bounds__(kThreads, 2) k_quantize8(const Quantize8Call c, Divide tiles_k, uint32_t tiles) {
  using M = Smem<T, VEC, COLS>;
  __shared__ __align__(16) float col_max[COLS ? kThreads / 32 : 1][kGroup8];
  __shared__ __align__(16) float col_inv[kGroup8];
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* const tile = smem + (M::RING ? M::DEPTH * M::STAGE : 0);
  wait_for_earlier_work();
  let_next_start();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this thread's units of a tile into the ring
  const auto fill = [&](uint32_t t, int stage) {
    if (t < tiles) {
      const uint32_t tr = quotient(tiles_k, t), tk = t - tr * tiles_k.d;
      const int64_t r = (int64_t)tr * kGroup8, k = (int64_t)tk * kGroup8;
      // rows and columns of the tile that there are (K is a multiple of 8)
      const int rows = (int)min((int64_t)kGroup8, c.R - r) - ty * kRows, cols = (int)min((int64_t)kGroup8, c.K - k) - tx * 8;
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem) + stage * M::STAGE + threadIdx.x * 16;
      const T* from = static_cast<const T*>(c.x) + (rows > 0 && cols > 0 ? (r + ty * kRows) * c.ld + k + tx * 8 : 0);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool on = i < rows && cols > 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * kThreads * 16), "l"(from),
                     "r"(on ? 16 : 0) : "memory");
        if (i + 1 < rows) from += c.ld;  // (an address in the matrix, whether it is read or not)
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (M::RING) {
#pragma unroll
    for (int k = 0; k < M::DEPTH - 1; ++k) fill(blockIdx.x + k * gridDim.x, k);
  }
  uint32_t step = 0;
#pragma unroll 1
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x, ++step) {
    const uint32_t tr = quotient(tiles_k, t), tk = t - tr * tiles_k.d;
    const int64_t tile_r = (int64_t)tr * kGroup8, tile_k = (int64_t)tk * kGroup8;
    const int rows_left = (int)min((int64_t)kGroup8, c.R - tile_r), cols_left = (int)min((int64_t)kGroup8, c.K - tile_k);
    const int64_t r0 = tile_r + ty * kRows, k0 = tile_k + tx * 8;
    const int nk = min(8, cols_left - tx * 8);          // this thread's columns (may be negative)
    const int nr = min(kRows, rows_left - ty * kRows);  // and rows
    float f[kRows][8];
    const T* x = static_cast<const T*>(c.x);
    if constexpr (M::RING) {
      fill(t + (M::DEPTH - 1) * gridDim.x, (step + M::DEPTH - 1) % M::DEPTH);
      asm volatile("cp.async.wait_group %0;" ::"n"(M::DEPTH - 1) : "memory");
      const T* from = reinterpret_cast<const T*>(smem + (step % M::DEPTH) * M::STAGE + threadIdx.x * 16);
#pragma unroll
      for (int i = 0; i < kRows; ++i) Load<T>::eight_shared(from + i * kThreads * 8, f[i]);
    } else if constexpr (VEC) {  // (K is a multiple of 8)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i < nr && nk > 0) {
          Load<T>::eight(x + (r0 + i) * c.ld + k0, f[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[i][e] = 0.f;
        }
      }
    } else {
      T* rows = reinterpret_cast<T*>(tile);
      constexpr int PER = kGroup8 / (kThreads / 32);  // rows of a warp
      T v[PER][4];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool on = warp * PER + i < rows_left;
        const T* from = x + (on ? (tile_r + warp * PER + i) * c.ld + tile_k + lane : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = on && lane + 32 * e < cols_left ? from[32 * e] : T(0.f);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) rows[(warp * PER + i) * Load<T>::PITCH + lane + 32 * e] = v[i][e];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRows; ++i) Load<T>::eight_shared(rows + (ty * kRows + i) * Load<T>::PITCH + tx * 8, f[i]);
    }
    // row maxima, and whether there is an infinity (in the warp's rows, or, where
    // columns need it, in the tile)
    float row[kRows];
    const auto row_maxima = [&] {
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        row[i] = max_abs8(f[i]);
        all = fmaxf(all, row[i]);
      }
      return all;
    };
    const bool infinite = row_maxima() > FLT_MAX;
    if (COLS ? __syncthreads_or(infinite) : __any_sync(0xffffffffu, infinite)) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = infinity_to_nan(f[i][e]);
      row_maxima();
    }
    float block = 0.f;
    if constexpr (COLS) {
      // column maxima: 4 rows of this thread, the other half of the warp, 16 warps
      float m8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m8[e] = max_abs3(f[0][e], f[1][e], max_abs3(f[2][e], f[3][e], 0.f));
        m8[e] = fmaxf(m8[e], __shfl_xor_sync(0xffffffffu, m8[e], 16));
      }
      // (each half of the warp stores half of a thread's columns)
      const bool high = lane >= 16;
      reinterpret_cast<float4*>(&col_max[warp][tx * 8])[high] =
          make_float4(high ? m8[4] : m8[0], high ? m8[5] : m8[1], high ? m8[6] : m8[2], high ? m8[7] : m8[3]);
      __syncthreads();
      if (threadIdx.x < kGroup8) {
        float m = col_max[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < kThreads / 32; ++k) m = fmaxf(m, col_max[k][threadIdx.x]);
        if (!c.blocks) {
          const uint32_t code = scale_code(m);
          m = scale_inverse(code);
          if ((int)threadIdx.x < cols_left)
            c.scales_t[(tile_k + threadIdx.x) * c.st_row + (int64_t)tr * c.st_group] = (uint8_t)code;
        }
        col_inv[threadIdx.x] = m;
      }
      __syncthreads();
      if (c.blocks) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, col_inv[lane + 32 * k]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t code = scale_code(m);
        block = scale_inverse(code);
        if (threadIdx.x == 0) c.scales[(int64_t)tr * c.s_row + (int64_t)tk * c.s_group] = (uint8_t)code;
      }
    }
    if (c.codes) {
      uint8_t* to = c.codes + (nr > 0 && nk > 0 ? r0 * c.ldc + k0 : 0);
      uint8_t* scale = c.scales + (nr > 0 ? (c.blocks ? 0 : r0 * c.s_row) + (int64_t)tk * c.s_group : 0);
#pragma unroll
      for (int i = 0; i < kRows; ++i, to += c.ldc, scale += c.s_row) {
        float inv = block;
        if (!COLS || !c.blocks) {
          float m = row[i];
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const uint32_t code = scale_code(m);
          inv = scale_inverse(code);
          if (tx == 0 && i < nr) *scale = (uint8_t)code;
        }
        if (i < nr && nk > 0)
          put_codes(to,
                    make_uint2(e4m3_four(f[i][0], f[i][1], f[i][2], f[i][3], inv),
                               e4m3_four(f[i][4], f[i][5], f[i][6], f[i][7], inv)), nk);
      }
    }
    if (COLS && c.codes_t) {
      // (every thread is past its reads of the tile as it came: the barriers above)
      const float4 lo = reinterpret_cast<const float4*>(col_inv)[2 * tx], hi = reinterpret_cast<const float4*>(col_inv)[2 * tx + 1];
      const float inv[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      uint8_t* const at = tile + tx * 8 * kGroup8 + ((ty ^ 2 * tx) << 2);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<uint32_t*>(at + e * kGroup8) =
            e4m3_four(f[0][e], f[1][e], f[2][e], f[3][e], c.blocks ? block : inv[e]);
      __syncthreads();
      // Eight threads write a column of the tile (128 bytes), 16 bytes each.  Odd
      // columns read their two halves in the other order: a warp's four columns
      // would otherwise be read from the same banks.
      const int word = (threadIdx.x & 7) * 4, left = rows_left - word * 4;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        const int col = pass * 64 + (threadIdx.x >> 3), turn = 2 * (col >> 3), odd = col & 1;
        const uint8_t* from = tile + col * kGroup8;
        uint2 a = *reinterpret_cast<const uint2*>(from + (((word + 2 * odd) ^ turn) << 2));
        uint2 b = *reinterpret_cast<const uint2*>(from + (((word + 2 - 2 * odd) ^ turn) << 2));
        if (odd) {
          const uint2 v = a;
          a = b;
          b = v;
        }
        if (col >= cols_left || left <= 0) continue;
        uint8_t* to = c.codes_t + (tile_k + col) * c.ldt + tile_r + word * 4;
        if (left >= 16) {
          *reinterpret_cast<uint4*>(to) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
          put_codes(to, a, min(8, left));
          if (left > 8) put_codes(to + 8, b, left - 8);
        }
      }
    }
  }
}

template <typename T, bool VEC, bool COLS>
cudaError_t launch(const Quantize8Call& c, uint32_t tiles, Divide tiles_k, cudaStream_t st) {
  using M = Smem<T, VEC, COLS>;
  auto kern = k_quantize8<T, VEC, COLS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)M::BYTES);
  uint32_t grid = tiles;
  if (e == cudaSuccess && M::RING) {  // persistent: two CTAs per SM
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    grid = std::min(tiles, 2u * (uint32_t)std::max(sms, 1));
  }
  if (e != cudaSuccess) return e;
  return launch_early(kern, grid, kThreads, M::BYTES, st, c, tiles_k, tiles);
}

template <typename T>
cudaError_t run(const Quantize8Call& c, cudaStream_t st) {
  const uint64_t tiles_k = (uint64_t)((c.K + kGroup8 - 1) / kGroup8);
  const uint64_t tiles = (uint64_t)((c.R + kGroup8 - 1) / kGroup8) * tiles_k;
  if (tiles > 0x3FFFFFFFull)  // (with the steps behind the last one in 32 bits)
    return cudaErrorInvalidConfiguration;
  const bool vec = c.K % 8 == 0 && reinterpret_cast<uintptr_t>(c.x) % 16 == 0 &&
                   c.ld * (int64_t)sizeof(T) % 16 == 0;
  const Divide tk = divide_by((uint32_t)tiles_k);
  const uint32_t n = (uint32_t)tiles;
  if (c.codes_t || c.blocks)
    return vec ? launch<T, true, true>(c, n, tk, st) : launch<T, false, true>(c, n, tk, st);
  return vec ? launch<T, true, false>(c, n, tk, st) : launch<T, false, false>(c, n, tk, st);
}

}  // namespace

cudaError_t quantize8(const Quantize8Call& c, bool f32, cudaStream_t st) {
  return f32 ? run<float>(c, st) : run<__nv_bfloat16>(c, st);
}

}  // namespace evo
