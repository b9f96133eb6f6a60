// wide.hpp -- a 256 x 256 tile of a product by eight waves, for results of many
// tiles (gated.hip): loads one and two steps ahead of the products, and the results
// taken from the accumulators without LDS, so that the next tile's first steps are
// loaded under this one's epilogue.
//
// Operands and their layouts in LDS are those of tile.hpp: a step of 64 along k is
// 32 KB of each operand.  All 160 KB of the CU's LDS hold three steps of the one
// operand and two of the other: at 64 bytes a cycle a step's 64 KB take a thousand
// cycles, which with the latency is as long as its products (2048 cycles), so that
// they do not all come in under the step before.  The direct loads to LDS
// are written in assembly: of the builtin's the compiler waits for all before the
// next read of LDS, also where that read is of another part.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"
#include "tile.hpp"

namespace oba {

namespace {

constexpr int kWideThreads = 512;
constexpr int kWideTile = 256;
constexpr int kWideHalf = kWideTile * kBK * 2;   // bytes of one operand's step
constexpr int kWideA = 3 * kWideHalf;             // the first operand's ring, then the second's
constexpr int kWideLds = kWideA + 2 * kWideHalf;

// A value that the compiler takes for a new one: what follows from it is worked out
// where it is used, and not kept in registers that the products need.
__device__ __forceinline__ uint32_t anew(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
  return v;
}

// The thread's number for one phase of a tile.
__device__ __forceinline__ uint32_t thread_anew() { return anew(threadIdx.x); }

// One thread's share of an operand of R rows in a block of NT threads, as Stage's
// of tile.hpp.
template <int SRC, int R, int NT>
struct AheadStage {
  static constexpr int P = R * (kBK / 8) / NT;
  uint32_t off[P];  // bytes from the step's origin

  __device__ __forceinline__ static uint32_t k_of(uint32_t i) {
    return SRC == kKRow ? ((i % (kBK / 8)) ^ (i / (kBK / 8) & 7u)) * 8 : i / (R / 8);
  }
  // r0: first row of the tile, of `rows`; rows past the last read the last
  __device__ __forceinline__ void init(uint32_t tid, int32_t r0, int32_t rows, uint32_t ld) {
    const uint32_t last = (uint32_t)(rows - 1 - r0);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t i = p * NT + tid, k = k_of(i);
      if constexpr (SRC == kKRow) {
        off[p] = (min(i / (kBK / 8), last) * ld + k) * 2;
      } else {
        const uint32_t c = i % (R / 8), block = kcol_block<R>(k, c / 2);
        off[p] = (k * ld + min(block * 16 + (c & 1) * 8, last & ~7u)) * 2;
      }
    }
  }

  // Pieces first .. first + n - 1 of a whole step straight to LDS, without a wait.
  // Five wait states lie between a vector instruction's write of a scalar register
  // (the buffer's) and a load that reads it, one between the write of m0 and the
  // load.  m0, which the compiler does not take as clobbered, is left as it was.
  __device__ __forceinline__ void ahead(int wave, const char* base, char* lds, int first = 0,
                                        int n = P) const {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __attribute__((address_space(3))) char* lp;
    typedef int i4 __attribute__((ext_vector_type(4)));
    const uint64_t b = (uint64_t)base;
    const i4 r = {(int)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                  (int)__builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xFFFFu)), -1,
                  0x00027000};
    const uint32_t to = (uint32_t)(uintptr_t)(lp)lds + wave * 1024u;
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (p >= first && p < first + n) {
        int m0;
        asm volatile(
            "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 2\n\t"
            "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
            : "=&s"(m0)
            : "s"(to + p * NT * 16), "v"(off[p]), "s"(r)
            : "memory");
      }
#endif
  }

  // A step of fewer than kBK elements through registers, 0 past them.
  __device__ __forceinline__ void tail(uint32_t tid, const char* base, char* lds,
                                       int32_t left) const {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int32_t k = (int32_t)k_of(p * NT + tid);
      lu4 u = {0u, 0u, 0u, 0u};
      if (k < left) {
        u = *reinterpret_cast<const lu4*>(global(base) + off[p]);
        if (SRC == kKRow && k + 8 > left) {
          for (int j = 0; j < 4; ++j)
            u[j] &= (k + 2 * j < left ? 0xFFFFu : 0u) | (k + 2 * j + 1 < left ? 0xFFFF0000u : 0u);
        }
      }
      *reinterpret_cast<lu4*>(lds + (p * NT + tid) * 16) = u;
    }
  }
};

// Where a wave's fragments lie in a step's operand, worked out once: the layouts of
// tile.hpp for rows row0 .. row0 + 16 n - 1, row0 a multiple of 64 (kKCol: n = 4).
// From fragment to fragment an address changes by a constant, added or, where the
// layout permutes, by exclusive or.
template <int SRC>
struct Frags;

template <>
struct Frags<kKRow> {
  uint32_t at;
  __device__ __forceinline__ void init(uint32_t row0) {
    const uint32_t l = threadIdx.x & 63, r = l & 15;
    at = (row0 + r) * 128u + (((l >> 4) ^ (r & 7u)) << 4);
  }
  __device__ __forceinline__ lu4 read(uint32_t lds, int ks, int i) const {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef const __attribute__((address_space(3))) lu4* lp;
    return *(lp)((anew(at) ^ (ks * 64u)) + lds + i * 2048u);
#else
    return lu4{0u, 0u, 0u, 0u};
#endif
  }
};

template <>
struct Frags<kKCol> {
  uint32_t at;
  __device__ __forceinline__ void init(uint32_t row0) {
    const uint32_t l = threadIdx.x & 63, k = (l >> 4) * 8 + ((l & 15) >> 2);
    at = kcol_at<kWideTile>(k, row0 >> 4) + (l & 3) * 8;
  }
  __device__ __forceinline__ lu4 read(uint32_t lds, int ks, int i) const {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __attribute__((address_space(3))) s4* lp;
    const uint32_t b = (anew(at) ^ (i * 32u)) + lds + ks * (32 * kWideTile * 2);
    const lu2 lo = __builtin_bit_cast(lu2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)b));
    const lu2 hi = __builtin_bit_cast(
        lu2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(b + 4 * kWideTile * 2)));
    return lu4{lo[0], lo[1], hi[0], hi[1]};
#else
    return lu4{0u, 0u, 0u, 0u};
#endif
  }
};

// All loads to LDS of this wave but the last LEFT have landed (loads come back in
// order; stores between them only make the wait longer).
template <int LEFT = 0>
__device__ __forceinline__ void wait_loads() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
#endif
}
// Every read of LDS of this wave has returned; all waves meet.
__device__ __forceinline__ void meet() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

// ---- across the four groups of 16 lanes ------------------------------------------
// Lane group g holds row l % 16's columns 4 g .. 4 g + 3 of a 16 x 16 tile.
// swap16 of a word each of two tiles: before, group g holds word g of both, after
// it words 2 (g / 2) and 2 (g / 2) + 1 of tile g % 2.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
#endif
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
#endif
}
// The largest of the four groups' values, in all of them.
__device__ __forceinline__ uint32_t max_groups(uint32_t v) {
  uint32_t w = v;
  swap16(v, w);
  v = w = max(v, w);
  swap32(v, w);
  return max(v, w);
}
// The four groups' words to all of them.
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&w)[4]) {
  w[0] = w[1] = v;
  swap16(w[0], w[1]);  // groups 0, 0, 2, 2 and 1, 1, 3, 3
  w[2] = w[0];
  w[3] = w[1];
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
}
// Transposes words of four tiles: before, group g holds word g of tiles 0 .. 3,
// after it words 0 .. 3 of tile g.  It is its own inverse.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
}

}  // namespace
}  // namespace oba
