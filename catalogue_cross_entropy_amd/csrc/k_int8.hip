// Scores of positions against items, both in 8 bits with a float32 scale per row (formula in
// include/rece.h): v_mfma_i32_32x32x32_i8, integer sums, one rounding of the scaled result.
//
// Bound by the results up to rows of some 256 bytes: 2,047 x 100,003 of bf16 are 409 MB.  Plain writes of that size reach
// 6.8 TB/s here, these 4.1 (4.7 where rows begin at whole lines of memory).  What matters is the order of the
// writes, more than what leads up to them: forms with the positions in registers and the items passing, through LDS
// or without, took 136 to 160 us, since they write to all rows at once.
//
// k_int8_march: rows of up to 256 bytes, see below.
//
// k_int8_tile: longer rows.  A workgroup of 4 waves forms a tile of 128 positions x 128 items, 128 bytes of each
// row at a time, the next 128 bytes' loads in flight during the products.  Items are the first
// operand, so a lane ends with four consecutive items of one position; the tile leaves through
// LDS in whole rows.  Neighbouring tiles (the same items, other positions) go to one XCD, whose L2
// then serves the items' rows and joins the ends of rows that neighbours write.  4,096 x 8,192 x 1,024: 57 us
// (1,200 Top/s).
//
// k_int8_few: up to 32 positions.  Bound by the items' rows, which are read once: every wave takes
// 32 items at a time straight from memory into the operand's registers.  5 x 1,000,000 x 128: 31 us (4.6 TB/s).
#include <algorithm>

#include "rece_device.h"
#include "rece_ops.h"
#include "rece_tile.h"

namespace rece {

constexpr int I8_T = 128;         // positions and items of a tile

int64_t int8_tiles(int64_t s, int64_t C) { return ((s + I8_T - 1) / I8_T) * ((C + I8_T - 1) / I8_T); }

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int I8_K = 128;         // bytes of a row at a time
constexpr int I8_FEW = 32;        // positions that k_int8_few takes
constexpr int I8_FEW_GRID = 2048; // its workgroups: eight per CU

struct Int8Args {
  const int8_t* x;
  const float* sx;
  const int8_t* y;
  const float* sy;
  void* out;
  int64_t s, C;
  int d;
  int nts;            // tiles along the positions (k_int8_march: workgroups along the items)
  int splits;         // k_int8_march: runs of positions
};

__device__ __forceinline__ i32x16 mma_i8(u32x4 a, u32x4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Four floats from the address of any one.
__device__ __forceinline__ f32x4 load_f4(const float* p) {
  struct __attribute__((packed, aligned(4))) Any {
    f32x4 v;
  };
  return reinterpret_cast<const Any*>(p)->v;
}

__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_one(bf16* p, float v) { p->bits = (uint16_t)pack_bf16(v, 0.0f); }

// 16 bytes to an address of any element.
template <int ALIGN>
__device__ __forceinline__ void store16(char* p, u32x4 v) {
  struct __attribute__((packed, aligned(ALIGN))) Any {
    u32x4 v;
  };
  reinterpret_cast<Any*>(p)->v = v;
}

// Rows of up to 32 KC bytes, more than 32 positions.  A wave holds 32 NI items in registers and goes over a run of
// positions, 32 at a time: block i multiplies the items NI n + i, so that lane n ends with NI consecutive items of a position
// and stores them at once, without LDS or waits for other waves.  All waves write the same few rows of results at a time:
// a memory page is filled while it is open.
template <class O, int KC, int NI>
__global__ __launch_bounds__(256, 2) void k_int8_march(Int8Args a) {
  constexpr int ES = sizeof(O), TI = 32 * NI;
  const int l = lane_id(), r = l & 31, hf = l >> 5;
  const int b = xcd_block(blockIdx.x, gridDim.x);
  const int64_t cw = (int64_t)(b % a.nts) * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t blocks = (a.s + 31) / 32, b0 = blocks * (b / a.nts) / a.splits, b1 = blocks * (b / a.nts + 1) / a.splits;
  const int64_t c = cw * TI + NI * r;                                    // the lane's first item
  if (cw * TI >= a.C) return;
  u32x4 fx[KC], fy[NI][KC];
  float sy[NI];
  const int end = a.d - 16;
#pragma unroll
  for (int i = 0; i < NI; ++i) {   // items beyond the end repeat the last one; 0 beyond the rows' end
    const int64_t m = min(c + i, a.C - 1);
    sy[i] = a.sy[m];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      fy[i][k] = u32x4{0u, 0u, 0u, 0u};
      if (32 * k + 16 * hf < a.d) fy[i][k] = *reinterpret_cast<const u32x4*>(a.y + m * a.d + 32 * k + 16 * hf);
    }
  }
  const int here = (int)max((int64_t)0, min((int64_t)NI, a.C - c));      // items of this lane
  float px[16];
  auto fetch = [&](int64_t bb) {   // positions beyond the end repeat the last one, chunks beyond a row's end its last one
    const int8_t* row = a.x + min(bb * 32 + r, a.s - 1) * a.d;
#pragma unroll
    for (int k = 0; k < KC; ++k) fx[k] = *reinterpret_cast<const u32x4*>(row + min(32 * k + 16 * hf, end));
  };
  if (b0 < b1) fetch(b0);
  for (int64_t bb = b0; bb < b1; ++bb) {
    const int64_t p0 = bb * 32;
#pragma unroll
    for (int v = 0; v < 16; ++v) px[v] = a.sx[min(p0 + tile_row(v) + 4 * hf, a.s - 1)];
    i32x16 acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      acc[i] = i32x16{};
#pragma unroll
      for (int k = 0; k < KC; ++k) acc[i] = mma_i8(fx[k], fy[i][k], acc[i]);
    }
    if (bb + 1 < b1) fetch(bb + 1);
    const int rows = (int)min((int64_t)32, a.s - p0);
    O* out = static_cast<O*>(a.out) + (p0 + 4 * hf) * a.C + c;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      if (tile_row(v) + 4 * hf >= rows) continue;
      float f[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) f[i] = (float)acc[i][v] * px[v] * sy[i];
      O* dst = out + tile_row(v) * a.C;
      if (here == NI) {
        struct __attribute__((packed, aligned(ES))) Piece {
          uint32_t w[NI * ES / 4];
        } o;
#pragma unroll
        for (int i = 0; i < NI * ES / 4; ++i)
          o.w[i] = ES == 2 ? pack_bf16(f[(2 * i) % NI], f[(2 * i + 1) % NI]) : __float_as_uint(f[i % NI]);
        *reinterpret_cast<Piece*>(dst) = o;
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (i < here) put_one(dst + i, f[i]);
      }
    }
  }
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
              *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
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

// KC > 0: rows of up to 32 KC bytes.  The positions stay in registers and the next 32 items' rows are on the way while
// these are multiplied.  KC = 0: longer rows, 128 bytes of both at a time.
template <class O, int KC>
__global__ __launch_bounds__(256) void k_int8_few(Int8Args a) {
  constexpr int N = KC ? KC : 4;
  const int l = lane_id(), r = l & 31, hf = l >> 5;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), waves = (int64_t)gridDim.x * 4;
  const int8_t* xr = a.x + min((int64_t)r, a.s - 1) * a.d + 16 * hf;
  const float px = a.sx[min((int64_t)r, a.s - 1)];
  const u32x4 none = {0u, 0u, 0u, 0u};
  u32x4 fx[N], fy[N];
  auto row_of = [&](int64_t b) { return a.y + min(b * 32 + r, a.C - 1) * a.d + 16 * hf; };
  auto load = [&](u32x4 (&f)[N], const int8_t* row, int k) {   // the second half of the last step may lie beyond the row
#pragma unroll
    for (int q = 0; q < N; ++q)
      f[q] = k + 32 * q + 16 * hf < a.d ? *reinterpret_cast<const u32x4*>(row + k + 32 * q) : none;
  };
  if constexpr (KC > 0) {
    load(fx, xr, 0);
    if (wave * 32 < a.C) load(fy, row_of(wave), 0);
  }
  for (int64_t b = wave; b * 32 < a.C; b += waves) {
    const int64_t c0 = b * 32;
    i32x16 acc = {};
    if constexpr (KC > 0) {
      u32x4 now[N];
#pragma unroll
      for (int q = 0; q < N; ++q) now[q] = fy[q];
      if ((b + waves) * 32 < a.C) load(fy, row_of(b + waves), 0);
#pragma unroll
      for (int q = 0; q < N; ++q) acc = mma_i8(now[q], fx[q], acc);
    } else {
      const int8_t* yr = row_of(b);
      for (int k = 0; k < a.d; k += 128) {
        load(fy, yr, k);
        load(fx, xr, k);
#pragma unroll
        for (int q = 0; q < N; ++q) acc = mma_i8(fy[q], fx[q], acc);
      }
    }
    if (r < a.s) {
      O* out = static_cast<O*>(a.out) + (int64_t)r * a.C;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = c0 + 8 * g + 4 * hf;
        float f[4];
        if (c + 4 <= a.C) {
          const f32x4 py = load_f4(a.sy + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = (float)acc[4 * g + e] * px * py[e];
          struct __attribute__((packed, aligned(sizeof(O)))) Out {
            u32x2_t v[sizeof(O) / 2];
          } o;
          if constexpr (sizeof(O) == 2) {
            o.v[0] = u32x2_t{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
          } else {
            o.v[0] = u32x2_t{__float_as_uint(f[0]), __float_as_uint(f[1])};
            o.v[1] = u32x2_t{__float_as_uint(f[2]), __float_as_uint(f[3])};
          }
          *reinterpret_cast<Out*>(out + c) = o;
        } else {
          for (int e = 0; e < 4; ++e)
            if (c + e < a.C) put_one(out + c + e, (float)acc[4 * g + e] * px * a.sy[c + e]);
        }
      }
    }
  }
}

template <class O>
hipError_t int8_launch(Int8Args a, hipStream_t st) {
  if (a.s <= I8_FEW) {
    const unsigned blocks = (unsigned)std::min<int64_t>((a.C + 127) / 128, I8_FEW_GRID);
    if (a.d <= 64) k_int8_few<O, 2><<<blocks, 256, 0, st>>>(a);
    else if (a.d <= 128) k_int8_few<O, 4><<<blocks, 256, 0, st>>>(a);
    else if (a.d <= 256) k_int8_few<O, 8><<<blocks, 256, 0, st>>>(a);
    else k_int8_few<O, 0><<<blocks, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  if (a.d <= 256) {
    // Four items to a lane while their rows fit in the registers (2,047 x 100,003 x 64: 105 us; two 112, eight 133),
    // and so many runs that two to three workgroups share a CU (d 64: 256 workgroups 139 us, 1,024 111, 2,048 105, 4,096
    // 120; d 128: 1,024 124, 2,048 132).
    const int TI = 128 * (a.d <= 128 ? 4 : 2);
    a.nts = (int)((a.C + TI - 1) / TI);
    const int64_t want = a.d <= 64 ? 2048 : 1024;
    a.splits = (int)std::max<int64_t>(1, std::min<int64_t>((want + a.nts - 1) / a.nts, (a.s + 31) / 32));
    const unsigned grid = (unsigned)(a.nts * a.splits);
    if (a.d <= 64) k_int8_march<O, 2, 4><<<grid, 256, 0, st>>>(a);
    else if (a.d <= 128) k_int8_march<O, 4, 4><<<grid, 256, 0, st>>>(a);
    else k_int8_march<O, 8, 2><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  a.nts = (int)((a.s + I8_T - 1) / I8_T);
  k_int8_tile<O><<<(unsigned)int8_tiles(a.s, a.C), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace


hipError_t int8_scores(bool bf16v, int64_t s, int64_t C, int d, const int8_t* x, const float* sx, const int8_t* y,
                       const float* sy, void* out, hipStream_t st) {
  const Int8Args a{x, sx, y, sy, out, s, C, d, 0, 0};
  return bf16v ? int8_launch<bf16>(a, st) : int8_launch<float>(a, st);
}

}  // namespace rece
