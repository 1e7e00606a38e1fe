// Matrix-core operands shared by the adapter and vocabulary kernels.
#pragma once

#include "common.hpp"

namespace f2i {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) v4s* lds_v4s_t;

// Two fp32 values as a pair of bf16, each rounded to nearest even (one instruction).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}

// One 16-byte operand per lane (row or column lane & 15, contraction group lane >> 4).
template <typename T> struct Mma;
template <> struct Mma<uint16_t> {
  static constexpr int kGroup = 8;     // contraction elements per lane and step
  __device__ static v4f run(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int kGroup = 4;
  __device__ static v4f run(v4u a, v4u b, v4f c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
};

// ds_read_b64_tr_b16: of 16 lanes, lane 4 i + q gives the address of columns 4 q .. 4 q + 3 of
// contraction row i, and lane l gets column l of the four rows.  (The restrict-qualified argument gives
// the read alias information; without any the compiler takes it to meet the copies in flight and waits
// for all of them first.)
__device__ __forceinline__ v2u read_transposed(lds_v4s_t __restrict p) {
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// One side of the product in LDS: ROWS rows by 128 bytes of contraction, 16-byte pieces permuted so that
// the lanes of an operand read cover all banks evenly.
//   Plain: row R at 128 R, its segment sg in place sg ^ (R % 8).
//   TRANS: contraction rows of ROWS elements as in memory; 16 columns of contraction row k (32 bytes of
//   bf16, 64 of fp32) lie in place unit ^ f(k), f(k) = k % 4 + 4 (k / 8 % 4) for bf16, k / 4 % 4 for
//   fp32: the sixteen (four) contraction rows of one read differ in f.
template <typename T, int ROWS, bool TRANS>
struct Side {
  static constexpr int kUnit = 16 * sizeof(T);            // bytes of 16 columns
  static constexpr int kUnits = ROWS / 16;
  __device__ static int f(int k) {
    return (sizeof(T) == 2 ? (k & 3) | (((k >> 3) & 3) << 2) : (k >> 2) & 3) & (kUnits - 1);
  }
  // Offset in memory (from the tile's first row, or the step's first contraction row and the tile's
  // first column) of the 16 bytes that lane `lane` of 1 KB copy `blk` brings.
  __device__ static uint32_t source(int blk, int lane, int64_t ld) {
    if constexpr (!TRANS) {
      const int R = blk * 8 + (lane >> 3), sg = (lane & 7) ^ (R & 7);
      return (uint32_t)(R * ld * sizeof(T)) + 16 * sg;
    } else {
      constexpr int kRow = ROWS * sizeof(T);
      const int pos = blk * 1024 + lane * 16, k = pos / kRow, in = pos % kRow;
      return (uint32_t)(k * ld * sizeof(T)) + ((in / kUnit) ^ f(k)) * kUnit + in % kUnit;
    }
  }
  // The lane's operand of 16-row fragment `frag` in half h of a step, at `base`.
  __device__ static __forceinline__ v4u read(const uint8_t* base, int frag, int h, int c, int g) {
    if constexpr (!TRANS) {
      return *reinterpret_cast<const v4u*>(base + (frag * 16 + c) * 128 + ((4 * h + g) ^ (c & 7)) * 16);
    } else if constexpr (sizeof(T) == 2) {
      constexpr int kRow = ROWS * 2;
      const int k = 8 * g + (c >> 2);
      const uint8_t* p = base + k * kRow + ((frag ^ f(k)) * kUnit) + (c & 3) * 8 + h * 32 * kRow;
      const v2u lo = read_transposed((lds_v4s_t)p), hi = read_transposed((lds_v4s_t)(p + 4 * kRow));
      return v4u{lo[0], lo[1], hi[0], hi[1]};
    } else {
      constexpr int kRow = ROWS * 4;
      const uint8_t* p = base + (16 * h + 4 * g) * kRow + ((frag ^ (g & (kUnits - 1))) * kUnit) + c * 4;
      return v4u{*reinterpret_cast<const uint32_t*>(p), *reinterpret_cast<const uint32_t*>(p + kRow),
                 *reinterpret_cast<const uint32_t*>(p + 2 * kRow), *reinterpret_cast<const uint32_t*>(p + 3 * kRow)};
    }
  }
};

}  // namespace f2i
