// out[m, n] = sum_k a[m, k] b[n, k] (+ add[m, n]), a and b in e4m3 with a
// power-of-two scale for each 128 elements along k (of one row, or of 128 rows),
// out in bf16 or fp32.
//
// The tensor core multiplies block-scaled operands on its own
// (kind::mxf8f6f4): a row's scale is a byte in tensor memory beside the
// accumulator, so the sum over all of K stays in tensor memory in fp32 and no
// CUDA core touches it before the end.  (The hardware's block is 32 elements; the
// four of a group of 128 get the same byte.  Its sums are rounded toward zero: off by
// 2.4e-7 in the root mean square over 4096 terms and 1.3e-6 over 16,384, below fp32's
// K 2^-24 and, for outputs in bf16, below their rounding.)
//
// One operand's rows lie on the 128 lanes of tensor memory (the M operand of the
// MMA), the other's on BQ of its columns (the N operand).  With many rows a's are
// on the lanes: a lane then holds consecutive columns of out, which go through a
// staging buffer per warp (32 rows of 128 bytes, 16-byte units XORed with the row)
// and leave in the widest units that out's base, row stride and width allow,
// whole rows of 128 bytes at a time.  (Stores straight from the registers of the
// other orientation, one element per lane, cost 500 instructions per 16 rows:
// 131 us for 147,456 x 512 fp32 outputs at K = 128.)  With few rows (up to 64
// tokens) b's are on the lanes, so that the MMA is no larger than the tokens (BQ
// down to 16) and b, the larger operand then, streams through the 128-row side;
// a warp stores 32 consecutive columns of a row.
//
// With long sums over many rows a wider tile of b pays (192 or 240 columns): a step of
// 128 k reads 46 KB for 128 x 240 products where 128 x 128 take 32, and each MMA
// instruction reads a's rows for more columns.  (240 and not 256: two accumulators and
// the scales share the 512 columns of tensor memory.)
//
// Long sums with few tiles are cut into pieces along k, one per CTA, which leave
// fp32 partial sums [piece][m][n], with b's rows on the lanes too; a second kernel
// adds them in order.
//
// Warps (384 or 640 threads, one persistent CTA per SM, a ring of stages of 128 k):
//   0      TMA producer: both operands' codes (128-byte swizzle)
//   1      MMA issuer: copies the scales of four (or two) groups to tensor memory
//          at a time, four MMAs of 32 k per group; commits free the stage
//   2, 3   scales of the two operands' rows: bytes from global memory, those of
//          the groups in a word (the MMA names the byte), in the order that the
//          copy to tensor memory wants (word r / 32 of 16-byte row r % 32)
//   4-...  epilogue: tensor memory -> registers -> out, two warps per lane
//          quarter taking alternate chunks of 128 bytes of a row; the accumulator
//          is double buffered, so the next tile's sum runs meanwhile, and with
//          short sums (up to 1024 k) each of the two has eight warps of its own
//          (147,456 x 128 outputs with an addend 50 -> 35 us, x 512 in fp32 64 -> 56)
//
// What it measures (device time): 589,824 x 516 at K = 128 146 us (69 % of the
// copy rate: the epilogue's latency; rows of 1032 bytes are stored 8 bytes at a
// time), 147,456 x 1024 at K = 128 65 us (72 %), 8192 x 4096 x 4096 117 us (2360
// TFLOP/s: 8 rounds of tiles of which 7.6 are needed, 32 steps of 0.46 us in each,
// the eighteenth tile of a row with 16 of 240 columns), 512 x 128 over 147,456 25 us,
// one row times 4096 x 1536 7 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "divide.cuh"
#include "launch.cuh"
#include "matmul8.h"
#include "sm103.h"
#include "tmap.h"

namespace evo {
namespace {

constexpr int kLanes = 128;  // rows of the operand on the lanes
constexpr int kGroup = 128;  // elements along k of a stage, and of a scale
enum Mode { kStaged, kDirect, kPartial };  // a on the lanes; b on the lanes; that, and a piece of the sum

// BQ: rows of the operand on the columns.  SETS: groups of eight epilogue warps.
template <int BQ_, Mode MODE, int SETS>
struct Cfg {
  static constexpr int BQ = BQ_;
  static constexpr bool WIDE = BQ > 128;  // scales of two blocks of 128 rows on the columns
  static constexpr int THREADS = 128 + SETS * 256;
  static constexpr uint32_t P_BYTES = kLanes * kGroup, Q_BYTES = BQ * kGroup;
  static constexpr uint32_t S_BYTES = 512;  // scales of up to 128 rows, four groups
  static constexpr uint32_t S_ENTRY = (WIDE ? 3 : 2) * S_BYTES;  // of p's rows, then q's
  static constexpr uint32_t STAGE = P_BYTES + Q_BYTES;
  // Scales: groups whose bytes go to tensor memory together (four fill a word;
  // fewer where 640 threads leave 96 registers, which bytes that are underway have
  // to fit: spilled, they are waited for), and such bundles requested ahead.
  static constexpr int BUNDLE = SETS == 1 ? 4 : 2, AHEAD = WIDE ? 2 : 3, RING_S = 4;
  static constexpr uint32_t STAGING = MODE == kStaged ? SETS * 8 * 4096 : 0;
  static constexpr int STAGES = std::min<int>(8, (int)((224 * 1024 - STAGING - RING_S * S_ENTRY) / STAGE));
  static constexpr uint32_t OFF_S = STAGES * STAGE;
  static constexpr uint32_t OFF_STAGING = OFF_S + RING_S * S_ENTRY;
  static constexpr uint32_t SMEM_ALLOC = OFF_STAGING + STAGING + 1024;
  // scales: 4 columns for each 128 rows, in as many places as there is room for, so that a
  // bundle is copied while the MMAs of those before it run (four instead of two: 1 % at
  // 36,864 x 1536, K = 384)
  static constexpr uint32_t COL_S = 2 * BQ < 32 ? 32 : 2 * BQ, COLS_S = WIDE ? 12 : 8;
  static constexpr int PLACES = WIDE ? 2 : 4;
  static_assert(PLACES <= RING_S && (RING_S & (RING_S - 1)) == 0, "the copy that a place waits for is in the ring");
  static_assert(COL_S + PLACES * COLS_S <= 512 && SMEM_ALLOC <= 227 * 1024, "tensor memory, shared memory");
  static_assert(STAGE % 1024 == 0 && OFF_STAGING % 1024 == 0, "the swizzle repeats every 1024 bytes");
};

struct Params8 {
  Operand8 p, q;          // on the lanes, on the columns
  int P, Q;               // their rows
  int groups, per_split, items;
  int fast_q;             // items run over q first
  Divide inner, outer;    // tiles along the axis that items run over first, and the other
  int M, N;
  void* out;
  int64_t ld_out;
  const void* add;
  int64_t ld_add;
  int unit, unit_add;     // bytes that out is stored, and add read, in at a time (staged)
  float* ws;
  WaitCfg wc;
};

// Instruction descriptor of kind::mxf8f6f4 with e4m3 operands, both K-major,
// E8M0 scales and fp32 accumulation.  Bits 4 and 5, and 29 and 30, say which byte
// of b's and a's scale words it takes.
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
  int p0, q0, g0, g1, split;
};
template <typename C>
__device__ __forceinline__ Item item_of(const Params8& p, int item) {
  Item w;
  const int t = (int)quotient(p.inner, item), i = item - t * (int)p.inner.d;
  w.split = (int)quotient(p.outer, t);
  const int o = t - w.split * (int)p.outer.d;
  w.p0 = (p.fast_q ? o : i) * kLanes;
  w.q0 = (p.fast_q ? i : o) * C::BQ;
  w.g0 = w.split * p.per_split;
  w.g1 = min(p.groups, w.g0 + p.per_split);
  return w;
}

// The scales of one operand's rows, RL for each lane: bytes from global memory
// into the ring that the MMA issuer copies to tensor memory.
template <typename C, int RL>
__device__ __forceinline__ void scale_role(const Params8& p, bool of_q, uint8_t* ring, uint64_t* bar_scale,
                                           uint64_t* bar_copied, const WaitCtx& wctx) {
  const Operand8 o = of_q ? p.q : p.p;
  const int rows = of_q ? p.Q : p.P, width = of_q ? C::BQ : kLanes;
  const int lane = threadIdx.x & 31;
  // A ring of bundles in registers: the bytes of one are requested AHEAD bundles
  // before they are written, across items too (requested one step ahead, every
  // step waited for L2: 950 cycles a step where its MMAs take 256).
  uint32_t s[C::AHEAD][RL][C::BUNDLE];
#pragma unroll
  for (int k = 0; k < C::AHEAD; ++k)
#pragma unroll
    for (int i = 0; i < RL; ++i)
#pragma unroll
      for (int j = 0; j < C::BUNDLE; ++j) s[k][i][j] = 0;  // (bytes of groups that there are not are not read)
  int item = (int)blockIdx.x, g = 0, g1 = 0;  // the bundle that is requested next
  const uint8_t* at[RL];  // where the rows' bytes lie; NULL for rows that there are not, whose scale is 1
  const auto enter = [&] {
    if (item >= p.items) return;
    const Item w = item_of<C>(p, item);
    g = w.g0;
    g1 = w.g1;
    const int r0 = of_q ? w.q0 : w.p0;
#pragma unroll
    for (int k = 0; k < RL; ++k) {
      const int r = lane + 32 * k;
      at[k] = r < width && r0 + r < rows ? o.scales + (int64_t)((r0 + r) >> o.shift) * o.s_row : nullptr;
    }
  };
  enter();
  const auto request = [&](uint32_t (&to)[RL][C::BUNDLE]) {
    if (item >= p.items) return;
    const int64_t off = g * o.s_group;
    const int n = min(C::BUNDLE, g1 - g);  // (the same for the whole warp)
#pragma unroll
    for (int j = 0; j < C::BUNDLE; ++j) {
      if (j >= n) break;
#pragma unroll
      for (int k = 0; k < RL; ++k) to[k][j] = at[k] ? at[k][off + j * o.s_group] : 127u;
    }
    g += C::BUNDLE;
    if (g >= g1) {
      item += (int)gridDim.x;
      enter();
    }
  };
  int left = 0;  // bundles of this CTA
  if (p.per_split >= p.groups) {  // (every item has all groups)
    left = (p.items - 1 - (int)blockIdx.x + (int)gridDim.x) / (int)gridDim.x *
           ((p.groups + C::BUNDLE - 1) / C::BUNDLE);
  } else {
    for (int i = (int)blockIdx.x; i < p.items; i += (int)gridDim.x) {
      const Item v = item_of<C>(p, i);
      left += (v.g1 - v.g0 + C::BUNDLE - 1) / C::BUNDLE;
    }
  }
#pragma unroll
  for (int k = 0; k < C::AHEAD; ++k) request(s[k]);
  bool ok = true;
  for (int is0 = 0; is0 < left && ok; is0 += C::AHEAD) {
#pragma unroll
    for (int k = 0; k < C::AHEAD; ++k) {
      const int is = is0 + k, slot = is % C::RING_S;
      if (is < left && ok) {
        uint32_t v[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) {
          v[i] = s[k][i][0];
#pragma unroll
          for (int j = 1; j < C::BUNDLE; ++j) v[i] |= s[k][i][j] << 8 * j;
        }
        if (is >= C::RING_S) ok = mbar_wait(&bar_copied[slot], ((is / C::RING_S) - 1) & 1, wctx);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
#pragma unroll
          for (int h = 0; h < RL / 4; ++h)
            *reinterpret_cast<uint4*>(ring + slot * C::S_ENTRY + ((of_q ? 1 : 0) + h) * C::S_BYTES + lane * 16) =
                make_uint4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
          fence_proxy_async_smem();  // generic writes, read by the copy to tensor memory
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_scale[slot]);
          request(s[k]);  // (behind the fence, which waits for loads that are underway)
        }
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ float load_one(const T* p);
template <>
__device__ __forceinline__ float load_one<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_one<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Shared memory by its own address (the compiler would take the generic one).
__device__ __forceinline__ uint4 lds(uint32_t at, uint4) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds(uint32_t at, uint2) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds(uint32_t at, uint32_t) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds(uint32_t at, uint16_t) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts(uint32_t at, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void sts(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void sts(uint32_t at, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
}

// Copies between a warp's staging buffer (rows of 128 bytes, 16-byte units XORed
// with the row) and 32 rows of a matrix, V bytes per lane.  `at`: the first row's
// first byte; `rows`, `width`: how many rows and bytes of a row there are (a
// multiple of V).  All of a lane's loads are issued before its stores (one after
// the other, each store behind its load, 147,456 x 128 outputs with an addend took
// 34 us).
template <int V>
struct Unit;
template <>
struct Unit<16> { using T = uint4; };
template <>
struct Unit<8> { using T = uint2; };
template <>
struct Unit<4> { using T = uint32_t; };
template <>
struct Unit<2> { using T = uint16_t; };

template <int V, bool STORE>
__device__ __forceinline__ void copy_rows(uint32_t stg, uint8_t* at, int64_t stride, int rows, int width) {
  using T = typename Unit<V>::T;
  constexpr int PER = 128 / V;                     // units of a row
  constexpr int STEP = PER <= 32 ? 32 / PER : 1;   // rows at a time
  constexpr int COUNT = 32 / STEP;                 // units of a lane
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int h = 0; h < (PER <= 32 ? 1 : PER / 32); ++h) {
    const int r0 = PER <= 32 ? lane / PER : 0, b = (PER <= 32 ? lane % PER : lane + 32 * h) * V;
    if (b >= width) continue;
    uint8_t* g = at + r0 * stride + b;
    const auto place = [&](int r) { return stg + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15); };
    T v[COUNT];
    if constexpr (STORE) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = lds(place(r0 + i * STEP), T{});
#pragma unroll
      for (int i = 0; i < COUNT; ++i, g += STEP * stride)
        if (r0 + i * STEP < rows) *reinterpret_cast<T*>(g) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < COUNT; ++i, g += STEP * stride) v[i] = r0 + i * STEP < rows ? *reinterpret_cast<const T*>(g) : T{};
#pragma unroll
      for (int i = 0; i < COUNT; ++i) sts(place(r0 + i * STEP), v[i]);
    }
  }
}
template <bool STORE>
__device__ __forceinline__ void copy_rows(int unit, uint32_t stg, uint8_t* at, int64_t stride, int rows, int width) {
  switch (unit) {
    case 16: return copy_rows<16, STORE>(stg, at, stride, rows, width);
    case 8: return copy_rows<8, STORE>(stg, at, stride, rows, width);
    case 4: return copy_rows<4, STORE>(stg, at, stride, rows, width);
    default: return copy_rows<2, STORE>(stg, at, stride, rows, width);
  }
}

// 128 bytes of a row of out for this lane: from the accumulator's columns to the
// lane's row of the staging buffer, with what the buffer holds of add.
__device__ __forceinline__ void stage_row(uint32_t stg, const uint32_t (&r)[32], bool add) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t to = stg + lane * 128 + ((c ^ (lane & 7)) << 4);
    uint4 v = make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
    if (add) {
      const uint4 a = lds(to, uint4{});
      v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(a.x));
      v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(a.y));
      v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(a.z));
      v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(a.w));
    }
    sts(to, v);
  }
}
__device__ __forceinline__ void stage_row(uint32_t stg, const uint32_t (&lo)[32], const uint32_t (&hi)[32], bool add) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t to = stg + lane * 128 + ((c ^ (lane & 7)) << 4);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(c < 4 ? lo[8 * c + e] : hi[8 * (c - 4) + e]);
    if (add) {
      const uint4 a = lds(to, uint4{});
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] += bf16lo(w[e]);
        f[2 * e + 1] += bf16hi(w[e]);
      }
    }
    sts(to, make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
  }
}

template <typename T, int BQ, Mode MODE, int SETS>
__global__ void __launch_bounds__(128 + SETS * 256, 1)
    k_matmul8(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q, const Params8 p) {
  using C = Cfg<BQ, MODE, SETS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bar_full[C::STAGES], bar_empty[C::STAGES], bar_scale[C::RING_S], bar_copied[C::RING_S], bar_done[2],
      bar_free[2], bar_drain, bar_never;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bar_full[i], 1);   // codes
      mbar_init(&bar_empty[i], 1);  // the stage's MMAs have read it
    }
    for (int i = 0; i < C::RING_S; ++i) {
      mbar_init(&bar_scale[i], 2);   // scales of both operands
      mbar_init(&bar_copied[i], 1);  // they are in tensor memory
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
  if (warp == 0 && lane == 0) { tma_prefetch_desc(&tm_p); tma_prefetch_desc(&tm_q); }
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
    for (int item = (int)blockIdx.x; item < p.items && ok; item += (int)gridDim.x) {
      const Item w = item_of<C>(p, item);
      for (int g = w.g0; g < w.g1; ++g, ++it) {
        const int st = it % C::STAGES;
        if (it >= C::STAGES) ok = mbar_wait(&bar_empty[st], ((it / C::STAGES) - 1) & 1, wctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_full[st], C::STAGE);
          tma_load_2d(smem + st * C::STAGE, &tm_p, &bar_full[st], g * kGroup, w.p0);
          tma_load_2d(smem + st * C::STAGE + C::P_BYTES, &tm_q, &bar_full[st], g * kGroup, w.q0);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      volatile int no_abort = 0;
      for (int i = max(0, it - C::STAGES); i < it; ++i)  // every copy lands before the CTA may exit
        mbar_wait(&bar_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================ MMA issuer ===============================
    constexpr uint32_t id = idesc_mxf8(128, BQ);
    const uint64_t dp0 = umma_desc(smem_u32(smem), 16, 1024, kSw128);
    const uint64_t dq0 = umma_desc(smem_u32(smem + C::P_BYTES), 16, 1024, kSw128);
    const uint64_t ds0 = umma_desc(smem_u32(smem + C::OFF_S), 16, 128, kSwNone);
    uint32_t sp = tmem + C::COL_S, sq = sp + 4;
    bool ok = true;
    int it = 0, is = 0, n = 0;
    for (int item = (int)blockIdx.x; item < p.items && ok; item += (int)gridDim.x, ++n) {
      const Item w = item_of<C>(p, item);
      const int buf = n & 1;
      if (n >= 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_free[buf], ((n >> 1) - 1) & 1, wctx));
        if (!ok) break;
      }
      tc_fence_after();
      for (int g = w.g0; g < w.g1; ++g, ++it) {
        const int st = it % C::STAGES, j = (g - w.g0) % C::BUNDLE;
        if (j == 0) {
          // The copy below goes over the scales of bundle is - PLACES, which its MMAs read.
          // Nothing orders a copy behind MMAs that were issued before it, but the commit
          // behind the next bundle's copy does: those MMAs precede it.  (Looked at before
          // the others, whose latency hides its own: waited for behind them, 589,824 x 516
          // at K = 128 took 152 us.)
          constexpr int NEXT = C::PLACES - 1;
          uint64_t* const read = &bar_copied[(is - NEXT) & (C::RING_S - 1)];
          const uint32_t turn = ((is - NEXT) / C::RING_S) & 1;
          const bool free = is <= NEXT || mbar_test(read, turn);
          ok = mbar_wait(&bar_scale[is % C::RING_S], (is / C::RING_S) & 1, wctx);
          if (!free) ok = ok && mbar_wait(read, turn, wctx);
          sp = tmem + C::COL_S + (is % C::PLACES) * C::COLS_S;
          sq = sp + 4;
        }
        ok = ok && mbar_wait(&bar_full[st], (it / C::STAGES) & 1, wctx);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dp = dp0 + ((uint32_t)(st * C::STAGE) >> 4), dq = dq0 + ((uint32_t)(st * C::STAGE) >> 4);
        if (elect_one()) {
          if (j == 0) {
            const uint64_t ds = ds0 + ((uint32_t)((is % C::RING_S) * C::S_ENTRY) >> 4);
            tmem_copy_scales(sp, ds);
            tmem_copy_scales(sq, ds + (C::S_BYTES >> 4));
            if constexpr (C::WIDE) tmem_copy_scales(sq + 4, ds + (2 * C::S_BYTES >> 4));
            umma_commit(&bar_copied[is % C::RING_S]);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_mxf8(tmem + buf * BQ, dp + 2 * kk, dq + 2 * kk, id | (uint32_t)j << 4 | (uint32_t)j << 29, sp, sq,
                      g > w.g0 || kk > 0 ? 1u : 0u);
          umma_commit(&bar_empty[st]);
          if (g + 1 == w.g1) umma_commit(&bar_done[buf]);
        }
        __syncwarp();
        if (j == 0) ++is;
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
    uint8_t* ring = smem + C::OFF_S;
    if constexpr (C::WIDE) {
      if (warp == 3)
        scale_role<C, 8>(p, true, ring, bar_scale, bar_copied, wctx);
      else
        scale_role<C, 4>(p, false, ring, bar_scale, bar_copied, wctx);
    } else {
      scale_role<C, 4>(p, warp == 3, ring, bar_scale, bar_copied, wctx);
    }
  } else {
    // ============================ epilogue =================================
    const int quad = warp & 3, half = (warp - 4) >> 2 & 1, set = (warp - 4) >> 3;
    bool ok = true;
    if (p.wc.stall) ok = __all_sync(0xffffffffu, stall_wait(&bar_never, wctx));
    int n = 0;
    for (int item = (int)blockIdx.x; item < p.items && ok; item += (int)gridDim.x, ++n) {
      const int buf = n & 1;
      if (SETS == 2 && buf != set) continue;  // the other set's
      const Item w = item_of<C>(p, item);
      ok = __all_sync(0xffffffffu, mbar_wait(&bar_done[buf], (n >> 1) & 1, wctx));
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + buf * BQ;
      // The accumulator is free for the next tile but one as soon as its values are
      // in registers.
      bool held = true;
      const auto release = [&] {
        tc_fence_before();
        mbar_arrive(&bar_free[buf]);
        held = false;
      };
      if constexpr (MODE == kStaged) {
        const uint32_t stg = smem_u32(smem + C::OFF_STAGING + (warp - 4) * 4096);
        constexpr int SPAN = 128 / sizeof(T);  // columns of a chunk
        const int m = w.p0 + quad * 32, rows = min(32, p.M - m);
#pragma unroll 1
        for (int c = half * SPAN; c < BQ; c += 2 * SPAN) {
          const int n = w.q0 + c, width = min(min(SPAN, BQ - c), p.N - n) * (int)sizeof(T);
          if (width <= 0 || rows <= 0) break;  // (the same for the whole warp)
          uint32_t lo[32], hi[32];
          tmem_ld32(base + c, lo);
          if constexpr (sizeof(T) == 2) tmem_ld32(base + c + 32, hi);
          __syncwarp();  // the previous chunk has left the buffer
          tmem_wait_ld();
          reg_fence32(lo);
          if constexpr (sizeof(T) == 2) reg_fence32(hi);
          if (c + 2 * SPAN >= BQ || n + 2 * SPAN >= p.N) release();
          if (p.add) {
            copy_rows<false>(p.unit_add, stg,
                             static_cast<uint8_t*>(const_cast<void*>(p.add)) + (m * p.ld_add + n) * (int64_t)sizeof(T),
                             p.ld_add * (int64_t)sizeof(T), rows, width);
            __syncwarp();
          }
          if constexpr (sizeof(T) == 2)
            stage_row(stg, lo, hi, p.add != nullptr);
          else
            stage_row(stg, lo, p.add != nullptr);
          __syncwarp();
          copy_rows<true>(p.unit, stg, static_cast<uint8_t*>(p.out) + (m * p.ld_out + n) * (int64_t)sizeof(T),
                          p.ld_out * (int64_t)sizeof(T), rows, width);
        }
      } else {
        const int col = w.p0 + quad * 32 + lane;  // this thread's column of out
        const bool on = col < p.N;
#pragma unroll 1
        for (int c = half; c < BQ / 16; c += 2) {
          const int m = w.q0 + c * 16, rows = min(16, p.M - m);
          if (rows <= 0) break;  // (the same for the whole warp)
          uint32_t r[16];
          tmem_ld16(base + c * 16, r);
          tmem_wait_ld();
          reg_fence16(r);
          if (c + 2 >= BQ / 16 || m + 32 >= p.M) release();
          if constexpr (MODE == kPartial) {
            float* to = p.ws + ((int64_t)w.split * p.M + m) * p.N + col;
#pragma unroll
            for (int i = 0; i < 16; ++i, to += p.N)
              if (i < rows && on) *to = __uint_as_float(r[i]);
          } else {
            T* to = static_cast<T*>(p.out) + m * p.ld_out + col;
            if (p.add) {
              const T* add = static_cast<const T*>(p.add) + m * p.ld_add + col;
#pragma unroll
              for (int i = 0; i < 16; ++i, add += p.ld_add)
                if (i < rows && on) r[i] = __float_as_uint(__uint_as_float(r[i]) + load_one<T>(add));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i, to += p.ld_out)
              if (i < rows && on) store_one(to, __uint_as_float(r[i]));
          }
        }
      }
      if (held) release();
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

// Adds the pieces of the sums: the eight warps of a CTA share 32 times V outputs,
// warp w takes the pieces w, w + 8, ..., so that a thread's few loads are in flight
// together, and the warps' sums are added in order.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    k_matmul8_sum(const float* ws, int splits, int64_t total, Divide n, T* out, int64_t ld_out, const T* add, int64_t ld_add) {
  using W = typename Unit<4 * V>::T;
  __shared__ float part[8][32 * V];
  wait_for_earlier_work();
  let_next_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = (int64_t)blockIdx.x * (32 * V), i = first + lane * V;
  float s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = 0.f;
  if (i < total) {
#pragma unroll 5
    for (int k = warp; k < splits; k += 8) {
      const W v = *reinterpret_cast<const W*>(ws + k * total + i);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += reinterpret_cast<const float*>(&v)[e];
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) part[warp][lane * V + e] = s[e];
  __syncthreads();
  if (threadIdx.x < 32 * V && first + threadIdx.x < total) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += part[k][threadIdx.x];
    const uint32_t at = (uint32_t)(first + threadIdx.x), m = quotient(n, at), col = at - m * n.d;
    if (add) v += load_one<T>(add + m * ld_add + col);
    store_one(out + m * ld_out + col, v);
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

// The widest unit in which rows of `width` bytes can be copied.
int unit_of(const void* p, int64_t stride, int64_t width) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(p) | (uint64_t)stride | (uint64_t)width;
  return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
}

template <typename T, int BQ, Mode MODE, int SETS = 1>
cudaError_t launch(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  using C = Cfg<BQ, MODE, SETS>;
  Params8 p{};
  p.p = MODE == kStaged ? c.a : c.b;
  p.q = MODE == kStaged ? c.b : c.a;
  p.P = MODE == kStaged ? c.M : c.N;
  p.Q = MODE == kStaged ? c.N : c.M;
  CUtensorMap tp, tq;
  if (!make_tmap_codes(&tp, p.p, p.P, c.K, kLanes) || !make_tmap_codes(&tq, p.q, p.Q, c.K, BQ)) {
    *tmap_ok = false;
    return cudaErrorInvalidValue;
  }
  p.fast_q = MODE == kStaged;  // out's columns first: the rows of a that are in flight are few
  p.inner = divide_by(p.fast_q ? pl.tiles_q : pl.tiles_p);
  p.outer = divide_by(p.fast_q ? pl.tiles_p : pl.tiles_q);
  p.groups = pl.groups; p.per_split = pl.per_split;
  p.items = pl.tiles_p * pl.tiles_q * pl.splits;
  p.M = c.M; p.N = c.N;
  p.out = c.out; p.ld_out = c.ld_out;
  p.add = c.add; p.ld_add = c.ld_add;
  const int64_t size = sizeof(T);
  p.unit = unit_of(c.out, c.ld_out * size, c.N * size);
  p.unit_add = unit_of(c.add, c.ld_add * size, c.N * size);
  p.ws = c.ws;
  p.wc = launch_wait(c.wait);
  auto kern = k_matmul8<T, BQ, MODE, SETS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)std::min(p.items, sms), C::THREADS, C::SMEM_ALLOC, st, tp, tq, p);
}

template <typename T>
cudaError_t launch_sum(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st) {
  const int64_t total = (int64_t)c.M * c.N;  // (below 2^31: a product in pieces has few tiles)
  const auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    return launch_early(k_matmul8_sum<T, V>, (unsigned)((total + 32 * V - 1) / (32 * V)), 256, 0, st, (const float*)c.ws,
                        pl.splits, total, divide_by((uint32_t)c.N), static_cast<T*>(c.out), c.ld_out,
                        static_cast<const T*>(c.add), c.ld_add);
  };
  // pieces are 16-byte aligned one after another; small sums keep the SMs busy
  return total % 4 == 0 && total >= 128 * (int64_t)sms ? go(std::integral_constant<int, 4>{})
                                                       : go(std::integral_constant<int, 1>{});
}

template <int BQ, int SETS>
cudaError_t staged(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  return c.f32 ? launch<float, BQ, kStaged, SETS>(c, pl, sms, st, tmap_ok)
               : launch<__nv_bfloat16, BQ, kStaged, SETS>(c, pl, sms, st, tmap_ok);
}

template <int BQ>
cudaError_t few_rows(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  if (pl.splits > 1) {
    const cudaError_t e = launch<float, BQ, kPartial>(c, pl, sms, st, tmap_ok);
    if (e != cudaSuccess) return e;
    return c.f32 ? launch_sum<float>(c, pl, sms, st) : launch_sum<__nv_bfloat16>(c, pl, sms, st);
  }
  return c.f32 ? launch<float, BQ, kDirect>(c, pl, sms, st, tmap_ok)
               : launch<__nv_bfloat16, BQ, kDirect>(c, pl, sms, st, tmap_ok);
}

}  // namespace

Matmul8Plan matmul8_plan(int M, int N, int K, int sms) {
  Matmul8Plan pl{};
  const auto tiles = [](int n, int by) { return (int)(((int64_t)n + by - 1) / by); };
  pl.groups = tiles(K, kGroup);
  // b's rows on the lanes, with the columns that a's few rows need
  pl.bq = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  pl.tiles_p = tiles(N, kLanes);
  pl.tiles_q = tiles(M, pl.bq);
  pl.splits = 1;
  pl.per_split = pl.groups;
  const int64_t count = (int64_t)pl.tiles_p * pl.tiles_q;
  if (2 * count <= sms && pl.groups > 16) {
    // Pieces of the sum, two groups at least, for as many CTAs as there are SMs.  On the
    // device, whole and in pieces, at 8, 12, 16, 24 and 32 groups: 1 x 4096 5.3 7.0 8.3 11.1
    // 13.8 and 5.0 5.3 5.6 6.7 7.4 us, 64 x 4096 5.8 7.4 8.9 11.8 14.6 and 6.9 7.2 7.6 8.6 9.3,
    // 100 x 1500 6.9 8.2 9.7 12.6 15.5 and 6.1 6.2 6.6 7.0 7.4.  The second launch costs a
    // call that is not captured 6 us of the host (24.5 instead of 18.5 at any of these
    // lengths).  The device alone would put the border at 8 to 12 groups; up to 16 a
    // captured call loses less than the other saves.
    const int64_t most = std::min<int64_t>(sms / count, pl.groups / 2);
    pl.per_split = (int)((pl.groups + most - 1) / most);
    pl.splits = (pl.groups + pl.per_split - 1) / pl.per_split;
  }
  if (M > 64 && pl.splits == 1) {  // a's rows on the lanes
    pl.staged = true;
    pl.bq = 128;
    if (pl.groups > 8) {
      // Long sums, where the epilogue is hidden: the width of the fewest rounds of all SMs
      // times what a step of 128 k takes, 0.40 us with 128 columns, 0.44 with 192, 0.48
      // with 240.  With 128, 192 and 240: 8192 x 4096 x 4096 177, 137 and 117 us, 4096^3
      // 91, 72, 62, 1300 x 4096 x 4096 41, 33, 34, 5000 x 400 x 3000 22.4, 16.3, 16.8,
      // 16,384 x 512 x 2048 30, 27, 28, 147,456 x 256 x 1152 66, 74, 80,
      // 2048 x 1024 x 1152 8.2, 10.3, 10.8.  (In bf16.  In fp32 with an addend the epilogue
      // still counts at 9 to 11 groups, where the choice is up to a quarter off:
      // 16,384 x 960 x 1152 39, 41, 49; 4096^3 96, 78, 72.)
      const auto cost = [&](int bq, int step) {
        return ((int64_t)tiles(M, kLanes) * tiles(N, bq) + sms - 1) / sms * step;
      };
      const int64_t by128 = cost(128, 20), by192 = cost(192, 22), by240 = cost(240, 24);
      if (std::min(by192, by240) < by128) pl.bq = by192 < by240 ? 192 : 240;
    }
    pl.tiles_p = tiles(M, kLanes);
    pl.tiles_q = tiles(N, pl.bq);
  }
  return pl;
}

size_t matmul8_workspace_bytes(int M, int N, int K, int sms) {
  const Matmul8Plan pl = matmul8_plan(M, N, K, sms);
  return pl.splits > 1 ? (size_t)pl.splits * M * N * sizeof(float) : 0;
}

cudaError_t matmul8(const Matmul8Call& c, const Matmul8Plan& pl, int sms, cudaStream_t st, bool* tmap_ok) {
  if (pl.staged) {
    if (pl.bq == 240) return staged<240, 1>(c, pl, sms, st, tmap_ok);
    if (pl.bq == 192) return staged<192, 1>(c, pl, sms, st, tmap_ok);
    return pl.groups <= 8 ? staged<128, 2>(c, pl, sms, st, tmap_ok) : staged<128, 1>(c, pl, sms, st, tmap_ok);
  }
  switch (pl.bq) {
    case 16: return few_rows<16>(c, pl, sms, st, tmap_ok);
    case 32: return few_rows<32>(c, pl, sms, st, tmap_ok);
    case 64: return few_rows<64>(c, pl, sms, st, tmap_ok);
    default:  // (only in pieces)
    {
      const cudaError_t e = launch<float, 128, kPartial>(c, pl, sms, st, tmap_ok);
      if (e != cudaSuccess) return e;
      return c.f32 ? launch_sum<float>(c, pl, sms, st) : launch_sum<__nv_bfloat16>(c, pl, sms, st);
    }
  }
}

}  // namespace evo
