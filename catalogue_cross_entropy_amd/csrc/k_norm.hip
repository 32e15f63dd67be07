// Root-mean-square norm of a residual stream after the addition of a branch, its gradients,
// and rows in 8 bits with a scale each (formulas in include/rece.h).  Bound by memory: every
// array is read or written once, in pieces of 8 elements (16 bytes of bf16) per lane.
//
// A row belongs to LPR lanes (a part of a wave, a wave, or a workgroup of 256) that hold NCH
// pieces each, so that a row is read once and its sum goes over few lanes.  Groups of lanes go
// over the rows with a stride and keep the weight in registers.
//
// Sums of squares are float64 (float32 squares pass the range from 1.8e19 on, and the additions
// hide behind the memory), and so are dweight's over a lane's rows, whose number grows with n (float32: 2.3 U sqrt(sum of the
// terms' squares) at 61 rows, now 1.1 U, U = 2^-24; 51,200 x 256 backward 17.2 -> 17.7 us).  Values in 8 bits are rint(127 p / max |p|), p = h w, decided as in
// float64: the float32 quotient decides where it is further from a half than its own error.
//
// Measured (bf16): 51,200 x 256 forward 17 us (105 MB, 6.1 TB/s with what the caches keep), backward 18 us and the join of
// the partial dweights 4 (float32: 40, 34, 5); 16,381 x 1,000 in 8 bits 25 us (115 MB, 4.6 TB/s; float32 40 us, 213 MB, 5.3);
// 5 x 64 in 8 bits 2.9 us, a launch.  Rows of a table in 8 bits, 1,000,000 x 128: 101 us (388 MB, 3.8 TB/s), where the
// float64 maximum and the rounding keep the vector unit 80 % busy at 3 bytes an element; float32 131 us (644 MB, 4.9 TB/s).
#include <algorithm>

#include "rece_device.h"
#include "rece_ops.h"
#include "rece_tile.h"

namespace rece {

namespace {

constexpr int NORM_THREADS = 256;
constexpr int NORM_GRID = 2048;        // workgroups that go over the rows: 8 per CU
constexpr int NORM_BWD_GRID = 1024;    // and in the backward pass, where each leaves a partial dweight

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 load8(const bf16* p) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
  F8 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r.v[2 * e] = __uint_as_float(w[e] << 16);
    r.v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ F8 load8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  F8 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r.v[e] = a[e];
    r.v[4 + e] = b[e];
  }
  return r;
}
__device__ __forceinline__ void store8(bf16* p, const F8& r) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack_bf16(r.v[2 * e], r.v[2 * e + 1]);
  *reinterpret_cast<u32x4*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const F8& r) {
  *reinterpret_cast<f32x4*>(p) = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
}
// the value as it is stored
__device__ __forceinline__ void rounded(F8& r, const bf16*) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = pack_bf16(r.v[2 * e], r.v[2 * e + 1]);
    r.v[2 * e] = __uint_as_float(w << 16);
    r.v[2 * e + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void rounded(F8&, const float*) {}

// Sum (or maximum) over the LPR lanes of a row, in every one of them.  Workgroup rows (LPR 256) go
// through `part`, 4 values of LDS; the caller separates two uses of the same values by a barrier.
template <int LPR, class F>
__device__ __forceinline__ double row_all(double v, F f, double* part) {
#pragma unroll
  for (int o = (LPR < 64 ? LPR : 64) / 2; o >= 1; o >>= 1) v = f(v, __shfl_xor(v, o));
  if constexpr (LPR == 256) {
    if (lane_id() == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = f(f(part[0], part[1]), f(part[2], part[3]));
  }
  return v;
}
__device__ __forceinline__ double add_d(double a, double b) { return a + b; }
// the larger one; NaN where one is
__device__ __forceinline__ double max_d(double a, double b) { return a > b || a != a ? a : b; }

// 1 / sqrt(v) as float32: float64 steps only where v itself leaves the range of float32
__device__ __forceinline__ float rstd_of(double v) {
  if (v > 1e-30 && v < 1e30) return 1.0f / sqrtf((float)v);
  return (float)(1.0 / sqrt(v));
}

enum NormMode { NORM_PLAIN = 0, NORM_INT8 = 1, QUANT_INT8 = 2 };

struct NormArgs {
  const void* x;
  const void* residual;   // or nullptr
  const float* weight;    // nullptr with QUANT_INT8
  void* h;                // or nullptr: not stored
  void* y;                // y (of the inputs' type) or int8
  float* rstd;            // [n], or the scales of int8 rows
  int64_t n;
  int d;
  float eps;
};

template <class E, int LPR, int NCH, int MODE>
__global__ __launch_bounds__(NORM_THREADS) void k_norm(NormArgs a) {
  constexpr int RPB = NORM_THREADS / LPR;   // rows of a workgroup at a time
  __shared__ double part[2][4];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int d = a.d, d8 = d >> 3;
  const double inv_d = 1.0 / d;
  F8 w[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int at = lane + c * LPR;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c].v[e] = MODE == QUANT_INT8 ? 1.0f : 0.0f;
    if (MODE != QUANT_INT8 && at < d8) w[c] = load8(a.weight + 8 * at);
  }
  // every lane of a workgroup makes the same number of rounds
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.n; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = r0 + sub;
    const bool live = r < a.n;
    const E* x = static_cast<const E*>(a.x) + r * d;
    const E* res = static_cast<const E*>(a.residual) + r * d;
    F8 h[NCH];
    double ss = 0.0, m = 0.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int at = lane + c * LPR;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c].v[e] = 0.0f;
      if (live && at < d8) {
        h[c] = load8(x + 8 * at);
        if (a.residual) {
          const F8 b = load8(res + 8 * at);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[c].v[e] += b.v[e];
          rounded(h[c], x);
        }
        if (a.h) store8(static_cast<E*>(a.h) + r * d + 8 * at, h[c]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (MODE != QUANT_INT8) ss = fma((double)h[c].v[e], (double)h[c].v[e], ss);
        if constexpr (MODE != NORM_PLAIN) m = max_d(m, fabs((double)h[c].v[e] * (double)w[c].v[e]));
      }
    }
    float rstd = 1.0f;
    if constexpr (MODE != QUANT_INT8) {
      ss = row_all<LPR>(ss, add_d, part[0]);
      rstd = rstd_of(ss * inv_d + (double)a.eps);
    }
    if constexpr (MODE == NORM_PLAIN) {
      if (live) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const int at = lane + c * LPR;
          if (at < d8) {
            F8 y;
#pragma unroll
            for (int e = 0; e < 8; ++e) y.v[e] = h[c].v[e] * rstd * w[c].v[e];
            store8(static_cast<E*>(a.y) + r * d + 8 * at, y);
          }
        }
        if (a.rstd && lane == 0) a.rstd[r] = rstd;
      }
      if (LPR == 256) __syncthreads();
    } else {
      m = row_all<LPR>(m, max_d, part[1]);
      // a row that holds a NaN or an infinity: scale NaN, values 0
      const bool ok = m < __builtin_huge_val();
      // 127 / m in float32 (0 where something might pass the range: then the float64 quotient decides)
      const float inv = m > 1e-30 && m < 1e30 ? (float)(127.0 / m) : 0.0f;
      if (live) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const int at = lane + c * LPR;
          if (at < d8) {
            uint32_t q[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float t = h[c].v[e] * w[c].v[e] * inv;
              float z = rintf(t);
              // t is off by at most 4 roundings of 127: 3.1e-5
              if (fabsf(fabsf(t - z) - 0.5f) < 1e-4f || inv == 0.0f)
                z = ok && m > 0.0 ? (float)rint(127.0 * ((double)h[c].v[e] * (double)w[c].v[e]) / m) : 0.0f;
              q[e >> 2] |= ((uint32_t)(int)z & 0xFFu) << (8 * (e & 3));
            }
            *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.y) + r * d + 8 * at) = make_uint2(q[0], q[1]);
          }
        }
        if (lane == 0) a.rstd[r] = !ok ? __builtin_nanf("") : m > 0.0 ? (float)(m * (double)rstd / 127.0) : 0.0f;
      }
      if (LPR == 256) __syncthreads();
    }
  }
}

struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* dh;        // or nullptr
  const float* weight;
  const float* rstd;
  void* dx;
  float* part;           // [grid][d] sums of dy h rstd over a workgroup's rows, rounded
  int64_t n;
  int d;
};

template <class E, int LPR, int NCH>
__global__ __launch_bounds__(NORM_THREADS) void k_norm_grad(NormGradArgs a) {
  constexpr int RPB = NORM_THREADS / LPR;
  __shared__ double part[4];
  extern __shared__ float sw[];   // [RPB][LPR * NCH * 8] where RPB > 1
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int d = a.d, d8 = d >> 3;
  F8 w[NCH];
  double dw[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int at = lane + c * LPR;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[c].v[e] = 0.0f;
      dw[c][e] = 0.0;
    }
    if (at < d8) w[c] = load8(a.weight + 8 * at);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.n; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = r0 + sub;
    const bool live = r < a.n;
    const float rstd = live ? a.rstd[r] : 0.0f;
    F8 h[NCH], g[NCH];
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int at = lane + c * LPR;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c].v[e] = g[c].v[e] = 0.0f;
      if (live && at < d8) {
        h[c] = load8(static_cast<const E*>(a.h) + r * d + 8 * at);
        g[c] = load8(static_cast<const E*>(a.dy) + r * d + 8 * at);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[c].v[e] *= rstd;                        // the normalised row
        dw[c][e] = fma((double)g[c].v[e], (double)h[c].v[e], dw[c][e]);
        g[c].v[e] *= w[c].v[e];
        s = fmaf(g[c].v[e], h[c].v[e], s);
      }
    }
    const float mean = (float)(row_all<LPR>((double)s, add_d, part) / d);
    if (live) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int at = lane + c * LPR;
        if (at < d8) {
          F8 o;
#pragma unroll
          for (int e = 0; e < 8; ++e) o.v[e] = rstd * fmaf(-h[c].v[e], mean, g[c].v[e]);
          if (a.dh) {
            const F8 b = load8(static_cast<const E*>(a.dh) + r * d + 8 * at);
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] += b.v[e];
          }
          store8(static_cast<E*>(a.dx) + r * d + 8 * at, o);
        }
      }
    }
    if (LPR == 256) __syncthreads();
  }
  float* out = a.part + (int64_t)blockIdx.x * d;
  F8 sum[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[c].v[e] = (float)dw[c][e];
  if constexpr (RPB == 1) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int at = lane + c * LPR;
      if (at < d8) store8(out + 8 * at, sum[c]);
    }
  } else {
    constexpr int W = LPR * NCH * 8;
#pragma unroll
    for (int c = 0; c < NCH; ++c) store8(sw + sub * W + 8 * (lane + c * LPR), sum[c]);
    __syncthreads();
    for (int t = threadIdx.x; t < d; t += NORM_THREADS) {
      double v = 0.0;
#pragma unroll
      for (int q = 0; q < RPB; ++q) v += (double)sw[q * W + t];
      out[t] = (float)v;
    }
  }
}

// out[t] = sum of the partial rows: 8 columns x 128 slices of the rows a workgroup.
__global__ __launch_bounds__(1024) void k_join_rows(const float* part, int rows, int d, float* out) {
  __shared__ double s[16][8];
  const int col = threadIdx.x & 7, slice = threadIdx.x >> 3, t = blockIdx.x * 8 + col;
  double v = 0.0;
  if (t < d) {
#pragma unroll 8
    for (int r = slice; r < rows; r += 128) v += (double)part[(int64_t)r * d + t];
  }
#pragma unroll
  for (int o = 32; o >= 8; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) < 8) s[threadIdx.x >> 6][col] = v;
  __syncthreads();
  if (threadIdx.x < 8 && t < d) {
    v = 0.0;
#pragma unroll
    for (int q = 0; q < 16; ++q) v += s[q][threadIdx.x];
    out[t] = (float)v;
  }
}

// f(lanes of a row, pieces of a lane): as few lanes as hold the row's pieces, up to a wave with 4 each.
template <class F>
hipError_t norm_shape(int d, F f) {
  const int d8 = d / 8;
  if (d8 <= 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  if (d8 <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (d8 <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (d8 <= 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  if (d8 <= 128) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (d8 <= 256) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  if (d8 <= 512) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
}

unsigned norm_grid(int64_t n, int rpb, int most) { return (unsigned)std::min<int64_t>((n + rpb - 1) / rpb, most); }

hipError_t launch_join(const float* part, int rows, int cols, float* out, hipStream_t st) {
  k_join_rows<<<(cols + 7) / 8, 1024, 0, st>>>(part, rows, cols, out);
  return hipGetLastError();
}

template <class E, int MODE>
hipError_t norm_launch(const NormArgs& a, hipStream_t st) {
  return norm_shape(a.d, [&](auto lpr, auto nch) {
    constexpr int LPR = decltype(lpr)::value, NCH = decltype(nch)::value;
    k_norm<E, LPR, NCH, MODE><<<norm_grid(a.n, NORM_THREADS / LPR, NORM_GRID), NORM_THREADS, 0, st>>>(a);
    return hipGetLastError();
  });
}

template <class E>
hipError_t norm_grad_launch(const NormGradArgs& a, float* dweight, hipStream_t st) {
  unsigned grid = 0;
  if (a.n == 0) return launch_join(nullptr, 0, a.d, dweight, st);
  const hipError_t e = norm_shape(a.d, [&](auto lpr, auto nch) {
    constexpr int LPR = decltype(lpr)::value, NCH = decltype(nch)::value, RPB = NORM_THREADS / LPR;
    grid = norm_grid(a.n, RPB, NORM_BWD_GRID);
    k_norm_grad<E, LPR, NCH><<<grid, NORM_THREADS, RPB == 1 ? 0 : RPB * LPR * NCH * 32, st>>>(a);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return launch_join(a.part, (int)grid, a.d, dweight, st);
}

}  // namespace

hipError_t launch_join_rows(const float* part, int rows, int cols, float* out, hipStream_t st) {
  return launch_join(part, rows, cols, out, st);
}

hipError_t norm_forward(bool bf16v, int64_t n, int d, float eps, const void* x, const void* residual, const float* weight,
                        void* h, void* y, float* rstd, hipStream_t st) {
  const NormArgs a{x, residual, weight, h, y, rstd, n, d, eps};
  return bf16v ? norm_launch<bf16, NORM_PLAIN>(a, st) : norm_launch<float, NORM_PLAIN>(a, st);
}

hipError_t norm_forward_int8(bool bf16v, int64_t n, int d, float eps, const void* x, const void* residual,
                             const float* weight, void* h, int8_t* y8, float* scale, hipStream_t st) {
  const NormArgs a{x, residual, weight, h, y8, scale, n, d, eps};
  return bf16v ? norm_launch<bf16, NORM_INT8>(a, st) : norm_launch<float, NORM_INT8>(a, st);
}

hipError_t quantize_rows(bool bf16v, int64_t n, int d, const void* x, int8_t* x8, float* scale, hipStream_t st) {
  const NormArgs a{x, nullptr, nullptr, nullptr, x8, scale, n, d, 0.0f};
  return bf16v ? norm_launch<bf16, QUANT_INT8>(a, st) : norm_launch<float, QUANT_INT8>(a, st);
}

size_t norm_workspace_bytes(int64_t n, int d) { return (size_t)std::min<int64_t>(n, NORM_BWD_GRID) * d * sizeof(float); }

hipError_t norm_backward(bool bf16v, int64_t n, int d, const void* dy, const void* h, const void* dh, const float* weight,
                         const float* rstd, void* ws, void* dx, float* dweight, hipStream_t st) {
  const NormGradArgs a{dy, h, dh, weight, rstd, dx, static_cast<float*>(ws), n, d};
  return bf16v ? norm_grad_launch<bf16>(a, dweight, st) : norm_grad_launch<float>(a, dweight, st);
}

}  // namespace rece
