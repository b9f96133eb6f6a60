// tile.hpp -- what the matrix products share (linear.hip, gated.hip): operands
// on their way from memory through LDS to the matrix instructions.
//
// Both compute C[r][c] = sum_k B(r, k) A(c, k) with the c side as the "A" operand
// of v_mfma_f32_16x16x32, so that a lane's four results are four consecutive
// columns of one row.  What differs is how an operand lies in memory:
//   kKRow   [r][k], k contiguous: kept so in LDS and read 16 bytes per lane
//   kKCol   [k][r], r contiguous: kept so in LDS and transposed by the
//           ds_read_b64_tr_b16 instruction while it is read
//   kKept   as kKCol with 8-bit elements, decoded to 16 bits (exactly) on the
//           way to LDS
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"
#include "layer_kernels.hpp"

namespace oba {

namespace {

enum Src { kKRow, kKCol, kKept };

constexpr int kBK = 64;  // the step along k: one 128-byte line of a kKRow operand's row

// ---- the matrix instruction ----------------------------------------------------
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ lf4 mfma(lu4 a, lu4 b, lf4 c, const _Float16*) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a),
                                                __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ lf4 mfma(lu4 a, lu4 b, lf4 c, const __bf16*) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                 __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// ---- LDS layouts -----------------------------------------------------------------
// kKRow: [R][kBK], 128 bytes a row, the 16-byte pieces of a row permuted by
// the row's low bits: the 16 rows that a fragment read touches at one k fall
// on all banks.  kKCol: [kBK][R], the 32-byte blocks of a row permuted by
// bits of k: a transposing read touches the 16 values of k that differ in
// bits 0-1 and 3-4, 32 bytes of each.
__device__ __forceinline__ uint32_t krow_at(uint32_t row, uint32_t piece) {
  return row * 128u + ((piece ^ (row & 7u)) << 4);
}
template <int R>
__device__ __forceinline__ uint32_t kcol_block(uint32_t k, uint32_t block) {
  const uint32_t f = (k & 3u) | ((k >> 3) & 3u) << 2;
  return (block ^ f) & (R / 16 - 1);
}
template <int R>
__device__ __forceinline__ uint32_t kcol_at(uint32_t k, uint32_t block) {
  return k * (R * 2u) + (kcol_block<R>(k, block) << 5);
}

// One thread's share of an operand's tile: pieces of 8 elements, each with a
// place of 16 bytes in LDS, places in the order of threads, so that a wave's
// 64 are one kilobyte: what the direct load from memory to LDS writes.  The
// permutation is therefore in the address that a place is loaded from.
// Rows past the operand's end read its last row (results there are not
// stored).
template <typename T, int SRC, int R, int NT>
struct Stage {
  static constexpr int P = R * (kBK / 8) / NT;
  static constexpr int kBytes = SRC == kKept ? 1 : 2;  // of an element in memory
  uint32_t off[P];   // bytes from the tile's origin
  uint32_t eoff[SRC == kKept ? P : 1];
  lu2 reg[SRC == kKept ? P : 1];  // kKept: a step's integers and exponents in flight
  uint32_t exp[SRC == kKept ? P : 1];

  // the k of piece p, from the step's first
  __device__ __forceinline__ static int32_t k_of(int p) {
    const uint32_t i = p * NT + threadIdx.x;
    if constexpr (SRC == kKRow)
      return (int32_t)((i % (kBK / 8)) ^ (i / (kBK / 8) & 7u)) * 8;
    else
      return (int32_t)(i / (R / 8));
  }

  // r0: first row of the tile, of `rows`; ld, eld: strides in elements
  __device__ __forceinline__ void init(int32_t r0, int32_t rows, uint32_t ld, uint32_t eld) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t i = p * NT + threadIdx.x;
      if constexpr (SRC == kKRow) {
        off[p] = (min(i / (kBK / 8), (uint32_t)(rows - 1 - r0)) * ld + (uint32_t)k_of(p)) * 2;
      } else {
        const uint32_t k = i / (R / 8), c = i % (R / 8);
        const uint32_t block = kcol_block<R>(k, c / 2);
        const uint32_t col = min(block * 16 + (c & 1) * 8, (uint32_t)(rows - 1 - r0) & ~7u);
        off[p] = (k * ld + col) * kBytes;
        if constexpr (SRC == kKept) eoff[p] = k * eld + col / kAct8Group;
      }
    }
  }

  // A whole step straight to LDS (16-bit operands): a buffer at the step's
  // origin, so that a lane's offsets never change.
  __device__ __forceinline__ void direct(const char* base, char* lds) const {
#if defined(__HIP_DEVICE_COMPILE__)  // the buffer type exists on the device only
    typedef __attribute__((address_space(3))) uint32_t* lp;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, -1, 0x00027000);
#pragma unroll
    for (int p = 0; p < P; ++p)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (lp)(lds + (p * NT + wave * 64) * 16), 16, off[p], 0, 0, 0);
#endif
  }

  // kKept: a step's elements to registers; at or past `left` they are 0.
  template <bool TAIL>
  __device__ __forceinline__ void load(const char* base, const uint8_t* ebase, int32_t left) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!TAIL || k_of(p) < left) {
        reg[p] = *reinterpret_cast<const lu2*>(base + off[p]);
        exp[p] = ebase[eoff[p]];
      } else {
        reg[p] = lu2{0u, 0u};
        exp[p] = 0u;
      }
    }
  }
  // An integer of at most 7 bits times a power of two: exact in T but for
  // binary16's range, which rows encoded from binary16 do not leave.
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float s = step_of(exp[p]);
      float v[8];
      for (int h = 0; h < 2; ++h) {
        uint32_t w = reg[p][h];
        // kept whole until here: the compiler took the bytes apart when they
        // were loaded and carried 32 registers from step to step
        asm("" : "+v"(w));
        for (int j = 0; j < 4; ++j) v[4 * h + j] = dequant(w, j, s);
      }
      *reinterpret_cast<lu4*>(lds + (p * NT + threadIdx.x) * 16) = pack(v, (const T*)nullptr);
    }
  }

  // The last step of a sum that is no multiple of kBK: through registers, the
  // elements past its end 0 (16-bit operands).
  __device__ __forceinline__ void tail(const char* base, char* lds, int32_t left) const {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int32_t k = k_of(p);
      lu4 u = {0u, 0u, 0u, 0u};
      if (k < left) {
        u = *reinterpret_cast<const lu4*>(base + off[p]);
        if (SRC == kKRow && k + 8 > left) {
          for (int j = 0; j < 4; ++j)
            u[j] &= (k + 2 * j < left ? 0xFFFFu : 0u) | (k + 2 * j + 1 < left ? 0xFFFF0000u : 0u);
        }
      }
      *reinterpret_cast<lu4*>(lds + (p * NT + threadIdx.x) * 16) = u;
    }
  }
};

// The fragment of 16 rows from `row` at k = 32 * ks: lane l holds row l % 16,
// k = 8 * (l / 16) .. +7.
template <int SRC, int R>
__device__ __forceinline__ lu4 fragment(const char* lds, uint32_t row, uint32_t ks) {
  const uint32_t l = threadIdx.x & 63;
  if constexpr (SRC == kKRow) {
    return *reinterpret_cast<const lu4*>(lds + krow_at(row + (l & 15), ks * 4 + (l >> 4)));
  } else {
    // the transposing read gives lane j of 16 the j-th column of a 4 x 16
    // block whose row i lies in lanes 4i .. 4i+3
    const uint32_t k = ks * 32 + (l >> 4) * 8 + ((l & 15) >> 2);
    typedef __attribute__((address_space(3))) s4* lp;
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lp)(lds + kcol_at<R>(k, row >> 4) + (l & 3) * 8));
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lp)(lds + kcol_at<R>(k + 4, row >> 4) + (l & 3) * 8));
    const lu2 a = __builtin_bit_cast(lu2, lo), b = __builtin_bit_cast(lu2, hi);
    return lu4{a[0], a[1], b[0], b[1]};
  }
}

// Eight results of row r from column c (c % 8 == 0).  n: columns from c to the
// last (may be more than 8, or none).  Rows of 16-bit operands hold memory up
// to a multiple of 8 columns.
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    *reinterpret_cast<lu4*>(p) = pack(v, (const T*)nullptr);
  } else {
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (T)v[j];
  }
}

// Blocks are handed to the 8 XCDs in turn; this gives each XCD a range of
// neighbouring tiles, so that its L2 sees an operand's rows once.
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
  const int64_t q = total / 8, r = total % 8, x = id % 8, i = id / 8;
  return x * q + min(x, r) + i;
}

// The 8 elements of a row from k; those at or past K are 0.
__device__ __forceinline__ lu4 load_k(const uint16_t* row, int64_t k, int64_t K) {
  if (k >= K) return lu4{0u, 0u, 0u, 0u};
  lu4 u = *reinterpret_cast<const lu4*>(row + k);
  if (k + 8 > K) {
    for (int j = 0; j < 4; ++j)
      u[j] &= (k + 2 * j < K ? 0xFFFFu : 0u) | (k + 2 * j + 1 < K ? 0xFFFF0000u : 0u);
  }
  return u;
}

}  // namespace
}  // namespace oba
