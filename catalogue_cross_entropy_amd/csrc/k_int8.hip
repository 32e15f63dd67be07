// Scores of positions against items, both in 8 bits with a float32 scale per row (formula in
// include/rece.h): v_mfma_i32_32x32x32_i8, integer sums, one rounding of the scaled result.
//
// k_int8_tile: a workgroup of 4 waves forms a tile of 128 positions x 128 items, 128 bytes of each
// row at a time, the next 128 bytes' loads in flight during the products.  Items are the first
// operand, so a lane ends with four consecutive items of one position; the tile leaves through
// LDS in whole rows.  Neighbouring tiles (the same items, other positions) go to one XCD, whose L2
// then serves the items' rows and joins the ends of rows that neighbours write.
//
// k_int8_few: up to 32 positions.  Bound by the items' rows, which are read once: every wave takes
// 32 items at a time straight from memory into the operand's registers.
#include <algorithm>

#include "rece_device.h"
#include "rece_internal.h"

namespace rece {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int I8_T = 128;         // positions and items of a tile
constexpr int I8_K = 128;         // bytes of a row at a time
constexpr int I8_FEW = 32;        // positions that k_int8_few takes

struct Int8Args {
  const int8_t* x;
  const float* sx;
  const int8_t* y;
  const float* sy;
  void* out;
  int64_t s, C;
  int d;
  int nts;            // tiles along the positions
  int64_t nt;         // tiles
};

__device__ __forceinline__ uint32_t pack_bf16_2(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

__device__ __forceinline__ i32x16 mma_i8(u32x4 a, u32x4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// 16 bytes to an address of any element.
template <int ALIGN>
__device__ __forceinline__ void store16(char* p, u32x4 v) {
  struct __attribute__((packed, aligned(ALIGN))) Any {
    u32x4 v;
  };
  reinterpret_cast<Any*>(p)->v = v;
}

template <class O>
__global__ __launch_bounds__(256, 2) void k_int8_tile(Int8Args a) {
  constexpr int CH = I8_K / 16;                       // 16-byte chunks of a row step
  constexpr int PT = I8_T * CH / 256;                 // chunks a thread copies of each side
  constexpr int SIDE = I8_T * I8_K;                   // bytes
  constexpr int ES = sizeof(O);
  constexpr int PITCH = I8_T * ES + 16;               // of a result row in LDS
  constexpr int LDS = 2 * SIDE > I8_T / 2 * PITCH ? 2 * SIDE : I8_T / 2 * PITCH;
  __shared__ __attribute__((aligned(16))) char smem[LDS];
  const int tid = threadIdx.x, wv = tid >> 6, l = lane_id(), r = l & 31, hf = l >> 5;
  const int wi = wv & 1, wp = wv >> 1;                // the wave's half of the items, of the positions
  const int64_t t = xcd_block(blockIdx.x, gridDim.x);
  const int64_t p0 = t % a.nts * I8_T, c0 = t / a.nts * I8_T;
  const int row = tid / CH, ch = tid % CH;            // rows row + 32 q
  const int swz = (ch ^ (row & 7)) << 4;
  u32x4 nx[PT], ny[PT];
  const int8_t* xr[PT];
  const int8_t* yr[PT];
#pragma unroll
  for (int q = 0; q < PT; ++q) {                      // rows beyond the end repeat the last one
    xr[q] = a.x + min(p0 + row + 32 * q, a.s - 1) * a.d + 16 * ch;
    yr[q] = a.y + min(c0 + row + 32 * q, a.C - 1) * a.d + 16 * ch;
  }
  auto fetch = [&](int k) {
    const bool in = k + 16 * ch < a.d;
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      nx[q] = in ? *reinterpret_cast<const u32x4*>(xr[q] + k) : u32x4{0u, 0u, 0u, 0u};
      ny[q] = in ? *reinterpret_cast<const u32x4*>(yr[q] + k) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  i32x16 acc[2][2] = {};   // [items][positions]
  fetch(0);
  for (int k = 0; k < a.d; k += I8_K) {
    if (k) __syncthreads();
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      *reinterpret_cast<u32x4*>(smem + (row + 32 * q) * I8_K + swz) = nx[q];
      *reinterpret_cast<u32x4*>(smem + SIDE + (row + 32 * q) * I8_K + swz) = ny[q];
    }
    __syncthreads();
    if (k + I8_K < a.d) fetch(k + I8_K);
    const int left = min(a.d - k, I8_K);
#pragma unroll
    for (int kk = 0; kk < I8_K / 32; ++kk) {
      if (kk * 32 >= left) break;
      const int c = ((2 * kk + hf) ^ (r & 7)) << 4;
      u32x4 fx[2], fy[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        fx[q] = *reinterpret_cast<const u32x4*>(smem + (64 * wp + 32 * q + r) * I8_K + c);
        fy[q] = *reinterpret_cast<const u32x4*>(smem + SIDE + (64 * wi + 32 * q + r) * I8_K + c);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) acc[i][p] = mma_i8(fy[i], fx[p], acc[i][p]);
    }
  }
  // scales: of the lane's two positions, and of its items 64 wi + 32 i + 8 (v / 4) + 4 hf + v % 4
  float px[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) px[p] = a.sx[min(p0 + 64 * wp + 32 * p + r, a.s - 1)];
  float py[2][16];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) py[i][v] = a.sy[min(c0 + 64 * wi + 32 * i + 8 * (v >> 2) + 4 * hf + (v & 3), a.C - 1)];
  const int wide = (int)min((int64_t)I8_T, a.C - c0);   // items of this tile
  constexpr int EPC = 16 / ES;                          // elements of a 16-byte piece
  constexpr int CPR = I8_T / EPC;                       // pieces of a row
#pragma unroll
  for (int half = 0; half < 2; ++half) {                // 64 positions at a time: those of the waves wp = half
    __syncthreads();
    if (wp == half) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = (float)acc[i][p][4 * g + e] * px[p] * py[i][4 * g + e];
            char* at = smem + (32 * p + r) * PITCH + (64 * wi + 32 * i + 8 * g + 4 * hf) * ES;
            if constexpr (ES == 2)
              *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16_2(f[0], f[1]), pack_bf16_2(f[2], f[3]));
            else
              *reinterpret_cast<f32x4*>(at) = f32x4{f[0], f[1], f[2], f[3]};
          }
    }
    __syncthreads();
    const int64_t q0 = p0 + 64 * half;
#pragma unroll 4
    for (int q = tid; q < 64 * CPR; q += 256) {
      const int rr = q / CPR, cc = q % CPR;
      if (q0 + rr < a.s) {
        char* dst = static_cast<char*>(a.out) + ((q0 + rr) * a.C + c0 + cc * EPC) * ES;
        const char* src = smem + rr * PITCH + cc * 16;
        if (cc * EPC + EPC <= wide) {
          store16<ES>(dst, *reinterpret_cast<const u32x4*>(src));
        } else {
          for (int e = 0; cc * EPC + e < wide; ++e)
            reinterpret_cast<O*>(dst)[e] = reinterpret_cast<const O*>(src)[e];
        }
      }
    }
  }
}

template <class O>
__global__ __launch_bounds__(256) void k_int8_few(Int8Args a) {
  const int l = lane_id(), r = l & 31, hf = l >> 5;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), waves = (int64_t)gridDim.x * 4;
  const int8_t* xr = a.x + min((int64_t)r, a.s - 1) * a.d + 16 * hf;
  const float px = a.sx[min((int64_t)r, a.s - 1)];
  for (int64_t b = wave; b * 32 < a.C; b += waves) {
    const int64_t c0 = b * 32;
    const int8_t* yr = a.y + min(c0 + r, a.C - 1) * a.d + 16 * hf;
    i32x16 acc = {};
#pragma unroll 4
    for (int k = 0; k < a.d; k += 32) {   // the second half of the last step may lie beyond the row
      const bool in = k + 16 * hf < a.d;
      const u32x4 fy = in ? *reinterpret_cast<const u32x4*>(yr + k) : u32x4{0u, 0u, 0u, 0u};
      const u32x4 fx = in ? *reinterpret_cast<const u32x4*>(xr + k) : u32x4{0u, 0u, 0u, 0u};
      acc = mma_i8(fy, fx, acc);
    }
    if (r < a.s) {
      O* out = static_cast<O*>(a.out) + (int64_t)r * a.C;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t c = c0 + 8 * (v >> 2) + 4 * hf + (v & 3);
        if (c < a.C) {
          const float f = (float)acc[v] * px * a.sy[c];
          if constexpr (sizeof(O) == 2)
            out[c].bits = (uint16_t)pack_bf16_2(f, 0.0f);
          else
            out[c] = f;
        }
      }
    }
  }
}

template <class O>
hipError_t int8_launch(Int8Args a, hipStream_t st) {
  if (a.s <= I8_FEW) {
    const int64_t blocks = (a.C + 127) / 128;
    k_int8_few<O><<<(unsigned)std::min<int64_t>(blocks, 4096), 256, 0, st>>>(a);
    return hipGetLastError();
  }
  a.nts = (int)((a.s + I8_T - 1) / I8_T);
  a.nt = a.nts * ((a.C + I8_T - 1) / I8_T);
  k_int8_tile<O><<<(unsigned)a.nt, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t int8_tiles(int64_t s, int64_t C) { return ((s + I8_T - 1) / I8_T) * ((C + I8_T - 1) / I8_T); }

hipError_t int8_scores(bool bf16v, int64_t s, int64_t C, int d, const int8_t* x, const float* sx, const int8_t* y,
                       const float* sy, void* out, hipStream_t st) {
  const Int8Args a{x, sx, y, sy, out, s, C, d, 0, 0};
  return bf16v ? int8_launch<bf16>(a, st) : int8_launch<float>(a, st);
}

}  // namespace rece
