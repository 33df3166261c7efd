// Counter-based random words for dropout masks that are never stored.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): four 32-bit words as a function of a
// 128-bit counter and a 64-bit key.  A mask row of C channels takes word c % 4
// of the block with the counter (c / 4, mask row, site, step) and the key seed,
// so that the forward and the backward pass, whatever their tiles, draw the
// same mask from (seed, step, site) alone.
//
// A block is 20 wide multiplications and as many logical operations for four
// elements.  At the memory rate of bf16 rows (read, add, write: four elements a
// cycle and SM) an SM would spend most of its issue slots on it: the residual add
// of 589,824 rows of 128 takes 89 us with a mask of its own for every row, where the
// bytes take 67 at the copy rate.  Rows that share a mask are therefore worked on
// together, with one draw (147,456 rows of 128: 20 us, 17 at the copy rate), and fp32 rows
// hide it (130 us, 133 at the copy rate, which is that of one read for each write).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace evo {

// The dropout of one call.
struct DropMask {
  const int64_t* rng;   // device: seed, step
  int64_t s[3];         // mask row index by (b, i, j); 0 along shared axes
  uint32_t site;
  uint32_t threshold;   // words from here on keep their element
  float scale;          // 1 / (1 - p)
};

struct PhiloxKey {
  uint32_t k0, k1, step, site;
};

__device__ __forceinline__ PhiloxKey philox_key(const DropMask& m) {
  const uint64_t seed = static_cast<uint64_t>(m.rng[0]);
  return PhiloxKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)m.rng[1], m.site};
}

__device__ __forceinline__ uint4 philox(const PhiloxKey& key, uint32_t group, uint32_t row) {
  uint32_t c0 = group, c1 = row, c2 = key.site, c3 = key.step, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Bit w: word w of the block keeps its element.
__device__ __forceinline__ uint32_t philox_keep4(const PhiloxKey& key, uint32_t threshold, uint32_t group,
                                                 uint32_t row) {
  const uint4 r = philox(key, group, row);
  return (r.x >= threshold ? 1u : 0u) | (r.y >= threshold ? 2u : 0u) | (r.z >= threshold ? 4u : 0u) |
         (r.w >= threshold ? 8u : 0u);
}

}  // namespace evo
