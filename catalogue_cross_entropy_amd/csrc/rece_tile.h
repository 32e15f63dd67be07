// Tiles of rows in LDS as operands of the 32 x 32 matrix-core products.
//
// A block of 32 x 32 products leaves lane l with column l % 32 and rows 8 (v / 4) + 4 (l / 32) + v % 4,
// v = 0 .. 15, which is also the operand layout of a second product over those rows (k = rows, in that
// order on both sides), so a block's values never leave their registers between two products; the rows
// enter the second one transposed through the LDS transpose read.
#pragma once
#include "rece_device.h"

namespace rece {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <class E> struct TileMma;
template <> struct TileMma<bf16> {
  static __device__ __forceinline__ f32x16 run(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct TileMma<float> {   // four coordinates per chunk and lane half: four products of depth 2
  static __device__ __forceinline__ f32x16 run(u32x4 a, u32x4 b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
};

// bf16 pair of two floats, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// LDS by byte offset: a per-lane offset and a constant that becomes the instruction's.
template <class T>
__device__ __forceinline__ T lds_at(uint32_t off) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>((uintptr_t)off);
}
__device__ __forceinline__ s16x4 lds_tr4(uint32_t off) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)off);
}
template <class T>
__device__ __forceinline__ void lds_put(uint32_t off, T v) {
  *reinterpret_cast<__attribute__((address_space(3))) T*>((uintptr_t)off) = v;
}

// Row of value v of a 32 x 32 block (less 4 h for the lane half h).
__device__ __forceinline__ constexpr int tile_row(int v) { return 8 * (v >> 2) + (v & 3); }

// Rows of D elements in LDS: 16-byte chunk c of row n is stored at chunk c ^ (n & SWM), which spreads the
// 32 rows a fragment read touches over the banks.
template <class E, int D> struct TileRows {
  static constexpr int RB = D * (int)sizeof(E);
  static constexpr int CPR = RB / 16;
  static constexpr int SWM = (CPR < 8 ? CPR : 8) - 1;
};

// Per-lane LDS offsets of a wave's fragment reads inside a tile.  The swizzle only mixes the low bits of
// a chunk's number, so a few offsets serve all reads, with constants added.
template <class E, int D> struct TileReads {
  using T = TileRows<E, D>;
  static constexpr int KC = T::RB / 32;
  static constexpr int NX = KC < (T::SWM + 1) / 2 ? KC : (T::SWM + 1) / 2;
  static constexpr int NY = sizeof(E) == 2 ? (D / 32 < 2 ? 1 : 2) : 4;
  uint32_t x[NX], y[NY];
  __device__ __forceinline__ void init() {
    const int l = lane_id(), h = l >> 5, r = l & 31;
#pragma unroll
    for (int k = 0; k < NX; ++k) x[k] = r * T::RB + (((2 * k + h) ^ (r & T::SWM)) << 4);
    if constexpr (sizeof(E) == 2) {
      // rows 4 h + j / 4, coordinates 16 ((l / 16) % 2) + 4 (j % 4) .. + 3 of each 32: within a 16-lane
      // group the transpose read hands lane i coordinate i of the group's four rows
      const int j = l & 15, half = (l >> 4) & 1, row = 4 * h + (j >> 2);
#pragma unroll
      for (int q = 0; q < NY; ++q)
        y[q] = row * T::RB + (((4 * q + 2 * half + ((j & 3) >> 1)) ^ (row & T::SWM)) << 4) + (j & 1) * 8;
    } else {
#pragma unroll
      for (int q = 0; q < NY; ++q) {
        const int row = 4 * h + q;
        y[q] = row * T::RB + (((r >> 2) ^ (row & T::SWM)) << 4) + 4 * (r & 3);
      }
    }
  }
  // 16-byte chunk 2 k + h of row l % 32
  static __device__ __forceinline__ u32x4 frag(const TileReads& o, uint32_t base, int k) {
    return lds_at<u32x4>(o.x[k % NX] + base + (k / NX) * (NX * 32));
  }
  // bf16: rows 16 kk .. 16 kk + 15 of the 32 at `base`, coordinates 32 nb + l % 32, in block order
  static __device__ __forceinline__ u32x4 across(const TileReads& o, uint32_t base, int nb, int kk) {
    const uint32_t at = o.y[nb % NY] + base + (nb / NY) * 128 + 16 * kk * T::RB;
    const s16x4 b[2] = {lds_tr4(at), lds_tr4(at + 8 * T::RB)};
    return __builtin_bit_cast(u32x4, b);
  }
  // float32: row tile_row(v) + 4 h, coordinate 32 nb + l % 32
  static __device__ __forceinline__ float across1(const TileReads& o, uint32_t base, int nb, int v) {
    return lds_at<float>(o.y[v & 3] + base + 8 * (v >> 2) * T::RB + nb * 128);
  }
};

}  // namespace rece
