// out[m, n] = sum_k a[m, k] b[n, k] (+ add[m, n]), a and b in e4m3 with a
// power-of-two scale for each 128 elements along k (of one row, or of 128 rows),
// out in bf16 or fp32.
//
// The tensor core multiplies block-scaled operands on its own
// (kind::mxf8f6f4): a row's scale is a byte in tensor memory beside the
// accumulator, so the sum over all of K stays in tensor memory in fp32 and no
// CUDA core touches it before the end.  (The hardware's block is 32 elements; the
// four of a group of 128 get the same byte.)
//
// A tile of out is 128 columns n, one per TMEM lane, and BM rows m, one per TMEM
// column: b's rows are the M = 128 operand of the MMA, a's rows the N = BM one.
// With the columns of out on the lanes a warp's store of one row is consecutive
// in memory, whatever out's stride and alignment, and few tokens (BM down to 16)
// cost no more tensor work than they have to, while b, the larger operand then,
// streams through the 128-row side.
//
// Long sums with few tiles are cut into pieces along k, one per CTA, which leave
// fp32 partial sums [piece][m][n]; a second kernel adds them in order.
//
// Warps (384 threads, one persistent CTA per SM, a ring of stages of 128 k):
//   0      TMA producer: a's and b's codes (128-byte swizzle)
//   1      MMA issuer: copies the stage's scales to tensor memory, four MMAs of
//          32 k; commits free the stage
//   2, 3   scales of b's and a's rows: bytes from global memory, each repeated
//          over a word, in the order that the copy to tensor memory wants
//          (word r / 32 of 16-byte row r % 32)
//   4-11   epilogue: tensor memory -> registers -> out, two warps per lane
//          quarter taking alternate chunks of 16 rows; the accumulator is double
//          buffered, so the next tile's sum runs meanwhile
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "matmul8.h"
#include "sm103.h"
#include "tmap.h"

namespace evo {
namespace {

constexpr int kLanes = 128;  // columns of out in a tile
constexpr int kGroup = 128;  // elements along k of a stage, and of a scale
constexpr int kThreads = 384;

template <int BM_>
struct Cfg {
  static constexpr int BM = BM_;
  static constexpr uint32_t B_BYTES = kLanes * kGroup, A_BYTES = BM * kGroup;
  static constexpr uint32_t S_BYTES = 512;  // scales of up to 128 rows
  static constexpr uint32_t STAGE = B_BYTES + A_BYTES;
  static constexpr int STAGES = std::min<int>(8, (200 * 1024) / (int)(STAGE + 2 * S_BYTES));
  static constexpr uint32_t OFF_S = STAGES * STAGE;
  static constexpr uint32_t SMEM_ALLOC = OFF_S + STAGES * 2 * S_BYTES + 1024;
  static constexpr uint32_t COL_S = 2 * BM < 32 ? 32 : 2 * BM;  // scales: 4 columns for b, 4 for a
  static_assert(COL_S + 8 <= 512, "tensor memory");
  static_assert(STAGE % 1024 == 0, "the swizzle repeats every 1024 bytes");
};

struct Params8 {
  Operand8 a, b;
  int M, N;
  int tiles_n, tiles_m, groups, per_split, items;
  void* out;
  int64_t ld_out;
  const void* add;
  int64_t ld_add;
  float* ws;
  WaitCfg wc;
};

// Instruction descriptor of kind::mxf8f6f4 with e4m3 operands, both K-major,
// E8M0 scales (byte 0 of each scale word) and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_mxf8(uint32_t M, uint32_t N) {
  return ((N >> 3) << 17) | (1u << 23) | ((M >> 7) << 27);
}
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                          uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// 32 rows of 16 bytes from shared memory to 4 columns of tensor memory, the same
// in each quarter of the lanes.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Where an item of work lies.
struct Item {
  int m0, n0, g0, g1, split;
};
__device__ __forceinline__ Item item_of(const Params8& p, int item, int bm) {
  Item w;
  const int t = item / p.tiles_n;
  w.n0 = (item - t * p.tiles_n) * kLanes;
  w.split = t / p.tiles_m;
  w.m0 = (t - w.split * p.tiles_m) * bm;
  w.g0 = w.split * p.per_split;
  w.g1 = min(p.groups, w.g0 + p.per_split);
  return w;
}

// Scale bytes of rows r0 + lane + 32 k (k < 4) of an operand for one group; rows
// that the operand does not have get 1.
__device__ __forceinline__ void scale_bytes(const Operand8& o, int rows, int r0, int width, int g, uint32_t (&s)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = lane + 32 * k;
    s[k] = r < width && r0 + r < rows
               ? o.scales[(int64_t)((r0 + r) >> o.shift) * o.s_row + (int64_t)g * o.s_group]
               : 127u;
  }
}

template <typename T>
__device__ __forceinline__ float load_one(const T* p);
template <>
__device__ __forceinline__ float load_one<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_one<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <typename T, int BM, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_matmul8(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Params8 p) {
  using C = Cfg<BM>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bar_full[C::STAGES], bar_scale[C::STAGES], bar_empty[C::STAGES], bar_done[2], bar_free[2],
      bar_drain, bar_never;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bar_full[i], 1);   // codes
      mbar_init(&bar_scale[i], 2);  // scales of a and of b
      mbar_init(&bar_empty[i], 1);  // the stage's MMAs have read it
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_done[i], 1);
      mbar_init(&bar_free[i], 256);  // the epilogue has read the accumulator
    }
    mbar_init(&bar_drain, 1);
    mbar_init(&bar_never, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, 512);
  if (warp == 0 && lane == 0) { tma_prefetch_desc(&tm_a); tma_prefetch_desc(&tm_b); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort_p = &abort_flag;
  const WaitCtx wctx{abort_p, p.wc};
  wait_for_earlier_work();
  let_next_start();

  if (warp == 0) {
    // ============================ codes ====================================
    bool ok = true;
    int it = 0;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
      const Item w = item_of(p, item, BM);
      for (int g = w.g0; g < w.g1; ++g, ++it) {
        const int st = it % C::STAGES;
        if (it >= C::STAGES) ok = mbar_wait(&bar_empty[st], ((it / C::STAGES) - 1) & 1, wctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_full[st], C::STAGE);
          tma_load_2d(smem + st * C::STAGE, &tm_b, &bar_full[st], g * kGroup, w.n0);
          tma_load_2d(smem + st * C::STAGE + C::B_BYTES, &tm_a, &bar_full[st], g * kGroup, w.m0);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {  // every copy lands before the CTA may exit
      volatile int no_abort = 0;
      for (int i = max(0, it - C::STAGES); i < it; ++i)
        mbar_wait(&bar_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================ MMA issuer ===============================
    constexpr uint32_t id = idesc_mxf8(128, BM);
    const uint64_t db0 = umma_desc(smem_u32(smem), 16, 1024, kSw128);
    const uint64_t da0 = umma_desc(smem_u32(smem + C::B_BYTES), 16, 1024, kSw128);
    const uint64_t ds0 = umma_desc(smem_u32(smem + C::OFF_S), 16, 128, kSwNone);
    const uint32_t sb = tmem + C::COL_S, sa = sb + 4;
    bool ok = true;
    int it = 0, n = 0;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x, ++n) {
      const Item w = item_of(p, item, BM);
      const int buf = n & 1;
      if (n >= 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_free[buf], ((n >> 1) - 1) & 1, wctx));
        if (!ok) break;
      }
      tc_fence_after();
      for (int g = w.g0; g < w.g1; ++g, ++it) {
        const int st = it % C::STAGES;
        ok = mbar_wait(&bar_full[st], (it / C::STAGES) & 1, wctx) &&
             mbar_wait(&bar_scale[st], (it / C::STAGES) & 1, wctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t db = db0 + ((uint32_t)(st * C::STAGE) >> 4), da = da0 + ((uint32_t)(st * C::STAGE) >> 4);
        const uint64_t ds = ds0 + ((uint32_t)(st * 2 * C::S_BYTES) >> 4);
        if (elect_one()) {
          tmem_copy_scales(sb, ds);
          tmem_copy_scales(sa, ds + (C::S_BYTES >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_mxf8(tmem + buf * BM, db + 2 * kk, da + 2 * kk, id, sb, sa, g > w.g0 || kk > 0 ? 1u : 0u);
          umma_commit(&bar_empty[st]);
          if (g + 1 == w.g1) umma_commit(&bar_done[buf]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(&bar_drain);
    __syncwarp();
    if (lane == 0) {
      volatile int no_abort = 0;
      mbar_wait(&bar_drain, 0, &no_abort);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ============================ scales ===================================
    const bool of_a = warp == 3;
    const Operand8 o = of_a ? p.a : p.b;
    const int rows = of_a ? p.M : p.N, width = of_a ? BM : kLanes;
    bool ok = true;
    int it = 0;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
      const Item w = item_of(p, item, BM);
      const int r0 = of_a ? w.m0 : w.n0;
      uint32_t s[4];
      scale_bytes(o, rows, r0, width, w.g0, s);
      for (int g = w.g0; g < w.g1; ++g, ++it) {
        const int st = it % C::STAGES;
        const uint4 v = make_uint4(s[0] * 0x01010101u, s[1] * 0x01010101u, s[2] * 0x01010101u, s[3] * 0x01010101u);
        if (g + 1 < w.g1) scale_bytes(o, rows, r0, width, g + 1, s);
        if (it >= C::STAGES) ok = mbar_wait(&bar_empty[st], ((it / C::STAGES) - 1) & 1, wctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        *reinterpret_cast<uint4*>(smem + C::OFF_S + (st * 2 + (of_a ? 1 : 0)) * C::S_BYTES + lane * 16) = v;
        fence_proxy_async_smem();  // generic writes, read by the copy to tensor memory
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_scale[st]);
      }
    }
  } else {
    // ============================ epilogue =================================
    const int quad = warp & 3, half = (warp - 4) >> 2;
    bool ok = true;
    if (p.wc.stall) ok = __all_sync(0xffffffffu, stall_wait(&bar_never, wctx));
    int n = 0;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x, ++n) {
      const Item w = item_of(p, item, BM);
      const int buf = n & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar_done[buf], (n >> 1) & 1, wctx));
      if (!ok) break;
      tc_fence_after();
      const int col = w.n0 + quad * 32 + lane;  // this thread's column of out
      const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + buf * BM;
#pragma unroll 1
      for (int c = half; c < BM / 16; c += 2) {
        const int m = w.m0 + c * 16;
        if (m >= p.M) break;  // (the same for the whole warp)
        uint32_t r[16];
        tmem_ld16(base + c * 16, r);
        tmem_wait_ld();
        reg_fence16(r);
        const int rows = min(16, p.M - m);
        if constexpr (SPLIT) {
          float* to = p.ws + ((int64_t)w.split * p.M + m) * p.N + col;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (i < rows && col < p.N) to[(int64_t)i * p.N] = __uint_as_float(r[i]);
        } else {
          const T* add = static_cast<const T*>(p.add) + m * p.ld_add + col;
          T* to = static_cast<T*>(p.out) + m * p.ld_out + col;
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[i] = __uint_as_float(r[i]);
            if (p.add && i < rows && col < p.N) f[i] += load_one<T>(add + i * p.ld_add);
          }
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < rows && col < p.N) to[i * p.ld_out] = f[i];
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < rows && col < p.N) to[i * p.ld_out] = __float2bfloat16_rn(f[i]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bar_free[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) report_abort(abort_p, p.wc);
}

// Adds the pieces of the sums in order.
template <typename T>
__global__ void __launch_bounds__(256)
    k_matmul8_sum(const float* ws, int splits, int M, int N, T* out, int64_t ld_out, const T* add, int64_t ld_add) {
  wait_for_earlier_work();
  let_next_start();
  const int64_t total = (int64_t)M * N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < splits; ++k) s += ws[k * total + i];
    const int64_t m = i / N, n = i - m * N;
    if (add) s += load_one<T>(add + m * ld_add + n);
    if constexpr (sizeof(T) == 4)
      out[m * ld_out + n] = s;
    else
      out[m * ld_out + n] = __float2bfloat16_rn(s);
  }
}

bool make_tmap_codes(CUtensorMap* map, const Operand8& o, int rows, int K, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ld};
  const cuuint32_t box[2] = {kGroup, box_rows}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(o.codes), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int BM, bool SPLIT>
cudaError_t launch(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  CUtensorMap ta, tb;
  if (!make_tmap_codes(&ta, c.a, c.M, c.K, BM) || !make_tmap_codes(&tb, c.b, c.N, c.K, kLanes)) {
    *tmap_ok = false;
    return cudaErrorInvalidValue;
  }
  Params8 p{};
  p.a = c.a; p.b = c.b;
  p.M = c.M; p.N = c.N;
  p.tiles_n = pl.tiles_n; p.tiles_m = pl.tiles_m;
  p.groups = pl.groups; p.per_split = pl.per_split;
  p.items = pl.tiles_n * pl.tiles_m * pl.splits;
  p.out = c.out; p.ld_out = c.ld_out;
  p.add = c.add; p.ld_add = c.ld_add;
  p.ws = c.ws;
  p.wc = launch_wait(c.wait);
  auto kern = k_matmul8<T, BM, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BM>::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  e = launch_early(kern, (unsigned)std::min(p.items, sms), kThreads, Cfg<BM>::SMEM_ALLOC, st, ta, tb, p);
  if (e != cudaSuccess || !SPLIT) return e;
  const int64_t blocks = ((int64_t)c.M * c.N + 255) / 256;
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, 8 * (int64_t)sms);
  return c.f32 ? launch_early(k_matmul8_sum<float>, grid, 256, 0, st, (const float*)c.ws, pl.splits, c.M, c.N,
                              static_cast<float*>(c.out), c.ld_out, static_cast<const float*>(c.add), c.ld_add)
               : launch_early(k_matmul8_sum<__nv_bfloat16>, grid, 256, 0, st, (const float*)c.ws, pl.splits, c.M,
                              c.N, static_cast<__nv_bfloat16*>(c.out), c.ld_out,
                              static_cast<const __nv_bfloat16*>(c.add), c.ld_add);
}

template <int BM>
cudaError_t by_type(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  if (pl.splits > 1) return launch<float, BM, true>(c, pl, sms, st, tmap_ok);
  return c.f32 ? launch<float, BM, false>(c, pl, sms, st, tmap_ok)
               : launch<__nv_bfloat16, BM, false>(c, pl, sms, st, tmap_ok);
}

}  // namespace

Matmul8Plan matmul8_plan(int M, int N, int K, int sms) {
  Matmul8Plan pl{};
  pl.bm = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  pl.tiles_m = (int)(((int64_t)M + pl.bm - 1) / pl.bm);
  pl.tiles_n = (int)(((int64_t)N + kLanes - 1) / kLanes);
  pl.groups = (int)(((int64_t)K + kGroup - 1) / kGroup);
  const int64_t tiles = (int64_t)pl.tiles_m * pl.tiles_n;
  int64_t splits = 1;
  if (2 * tiles <= sms) splits = std::min<int64_t>(sms / tiles, std::max(1, pl.groups / 2));
  pl.per_split = (int)((pl.groups + splits - 1) / splits);
  pl.splits = (pl.groups + pl.per_split - 1) / pl.per_split;
  return pl;
}

size_t matmul8_workspace_bytes(int M, int N, int K, int sms) {
  const Matmul8Plan pl = matmul8_plan(M, N, K, sms);
  return pl.splits > 1 ? (size_t)pl.splits * M * N * sizeof(float) : 0;
}

cudaError_t matmul8(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  switch (pl.bm) {
    case 16: return by_type<16>(c, pl, sms, st, tmap_ok);
    case 32: return by_type<32>(c, pl, sms, st, tmap_ok);
    case 64: return by_type<64>(c, pl, sms, st, tmap_ok);
    default: return by_type<128>(c, pl, sms, st, tmap_ok);
  }
}

}  // namespace evo
