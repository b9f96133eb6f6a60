// philox.hpp -- the dropout's random bits: Philox4x32 with 10 rounds (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).
// A counter of four words goes through ten rounds of two 32 x 32 -> 64 bit
// products keyed by two words; any counter can be had at any time, so a mask is
// never stored: the backward pass computes it again.
//
// The counter is (number of the block of eight columns, 64 bits; site; step):
// block row * ceil(cols / 8) + col / 8 of the matrix, one word that tells the
// dropouts of a step apart and one that tells the steps apart.  An element has
// 16 of the 128 bits: column col of a block of eight those of word (col % 8) /
// 2, the lower half first.  It is kept if they reach the threshold t = rate *
// 65536 rounded to nearest, and then multiplied by 65536 / (65536 - t), so that
// the expected value is exact for the rate as it is rounded.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"
#include "sublayer_kernels.hpp"

namespace oba {

namespace {

struct RngKey {
  uint32_t k0, k1, step;
};

// What lies on the device: seed and step.
__device__ __forceinline__ RngKey load_key(const Dropout& d) {
  RngKey k{0u, 0u, 0u};
  if (d.threshold) {
    const uint64_t seed = d.rng[0], step = d.rng[1];
    auto uniform = [](uint64_t v) {
      return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    };
    k = RngKey{uniform(seed), uniform(seed >> 32), uniform(step)};
  }
  return k;
}

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
#else
  return a ^ b ^ c;
#endif
}

__device__ __forceinline__ lu4 philox(uint64_t block, uint32_t site, const RngKey& key) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = site, c3 = key.step;
  uint32_t k0 = key.k0, k1 = key.k1;
#if defined(__HIP_DEVICE_COMPILE__)
  // each round's key is made where it is used: 20 of them kept over a loop of rows
  // pushed other scalars out of their registers
  asm volatile("" : "+s"(k0), "+s"(k1));
#endif
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = xor3((uint32_t)(b >> 32), c1, k0);
    c2 = xor3((uint32_t)(a >> 32), c3, k1);
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return lu4{c0, c1, c2, c3};
}

// Drops or scales the lane's V columns from column col of a row: eight are a
// block, four are one half of a block.  A dropped element is 0 whatever it was.
template <int V>
__device__ __forceinline__ void drop(const Dropout& d, const RngKey& key, int64_t row,
                                     int32_t blocks, int32_t col, float (&v)[V]) {
  static_assert(V == 4 || V == 8, "16 bytes of a row");
  const lu4 w = philox((uint64_t)(row * blocks + col / 8), d.site, key);
  const uint32_t t = d.threshold << 16;
#pragma unroll
  for (int j = 0; j < V; j += 2) {
    const uint32_t u = V == 8 ? w[j / 2] : (col & 4) ? w[2 + j / 2] : w[j / 2];
    v[j] = (u << 16) >= t ? v[j] * d.scale : 0.0f;
    v[j + 1] = (u | 0xFFFFu) >= t ? v[j + 1] * d.scale : 0.0f;
  }
}

}  // namespace
}  // namespace oba
