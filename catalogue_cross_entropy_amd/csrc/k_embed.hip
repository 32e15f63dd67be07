// Item embedding: rows of the item table as a model's inputs, and the table's gradient.
//   forward   out_i = scale * table[ids_i]  (padding ids: zero rows)
//   backward  dtable_j = scale * sum over i with ids_i = j of dout_i
// Both are bound by memory.  Rows move as 16-byte pieces: LPR lanes (a power of two)
// per row, 64 / LPR rows per wave instruction, several rows in flight per lane group.
// The backward pass sorts (id, i) by id (stable), cuts the sorted records into fixed
// pieces and sums each piece's runs in float32 registers; a run inside one piece is
// written at once, a run over several pieces leaves one partial row per piece that a
// second kernel adds in a fixed order, so every result is reproducible bit for bit.
#include <algorithm>

#include "rece_device.h"
#include "rece_internal.h"
#include "rece_parts.h"

namespace rece {

namespace {

constexpr int EMB_THREADS = 256;
constexpr int EMB_PIECE = 8;    // sorted records per piece

template <class E> struct Piece16 {
  static constexpr int EPL = 16 / (int)sizeof(E);
};

// Sixteen bytes of a row as floats, and back.
__device__ __forceinline__ void unpack16(u32x4 u, float (&v)[8]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    v[2 * t] = __uint_as_float(u[t] << 16);
    v[2 * t + 1] = __uint_as_float(u[t] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack16(u32x4 u, float (&v)[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) v[t] = __uint_as_float(u[t]);
}
// Round to nearest even; a NaN stays a NaN (its payload's low half could carry into infinity).
__device__ __forceinline__ uint32_t bf16_of(float x) { return x != x ? 0x7FC0u : bf16_bits_rne(x); }
__device__ __forceinline__ u32x4 pack16(const float (&v)[8]) {
  u32x4 u;
#pragma unroll
  for (int t = 0; t < 4; ++t) u[t] = bf16_of(v[2 * t]) | (bf16_of(v[2 * t + 1]) << 16);
  return u;
}
__device__ __forceinline__ u32x4 pack16(const float (&v)[4]) {
  return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}

// ------------------------------------------------------------------ forward
template <class E, int LPR>
__global__ __launch_bounds__(EMB_THREADS) void k_embed_rows(const E* __restrict__ table, const int32_t* __restrict__ ids,
                                                            E* __restrict__ out, int64_t n, int64_t C, int d, float scale) {
  constexpr int EPL = Piece16<E>::EPL;
  constexpr int RPI = WAVE / LPR;
  constexpr int UNR = 4;
  const int l = lane_id(), q = l / LPR;
  const int col = ((int)blockIdx.y * LPR + l % LPR) * EPL;
  if (col >= d) return;
  const int64_t r0 = ((int64_t)blockIdx.x * (EMB_THREADS / WAVE) + (threadIdx.x >> 6)) * (RPI * UNR) + q;
  int id[UNR];
  u32x4 raw[UNR];
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    const int64_t r = r0 + u * RPI;
    id[u] = r < n ? ids[r] : -1;
  }
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    const bool ok = id[u] >= 0 && id[u] < C;
    raw[u] = u32x4{0u, 0u, 0u, 0u};
    if (ok) raw[u] = *reinterpret_cast<const u32x4*>(table + (int64_t)id[u] * d + col);
    if (!ok) id[u] = -1;
  }
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    const int64_t r = r0 + u * RPI;
    if (r >= n) continue;
    float v[EPL];
    unpack16(raw[u], v);
#pragma unroll
    for (int t = 0; t < EPL; ++t) v[t] = id[u] < 0 ? 0.0f : v[t] * scale;   // a zero row, whatever scale is
    *reinterpret_cast<u32x4*>(out + r * d + col) = pack16(v);
  }
}

// ------------------------------------------------------------------ backward
__global__ __launch_bounds__(EMB_THREADS) void k_embed_clear(u32x4* __restrict__ p, int64_t n16) {
  const int64_t step = (int64_t)gridDim.x * EMB_THREADS;
  for (int64_t t = (int64_t)blockIdx.x * EMB_THREADS + threadIdx.x; t < n16; t += step) p[t] = u32x4{0u, 0u, 0u, 0u};
}

struct EmbGrad {
  const int32_t* K;        // sorted ids
  const int32_t* V;        // their rows (bit 31 set)
  const uint32_t* ntot;    // records
  const void* dout;
  const float* weight;     // per row, every wstride-th, or NULL
  int wstride;
  SweepParts parts;        // partial rows added first (rows NULL: none)
  float* partial;          // [pieces][2][d]: the piece's part of a run that began earlier, and of one that goes on
  void* dtable;
  int d;
  float scale;
  int b16, acc;
};

// EPL values of row j: written, or added (accumulate: the only writer of the row in this call).
template <int EPL>
__device__ __forceinline__ void put_row(const EmbGrad& a, int64_t j, int col, float (&v)[EPL]) {
#pragma unroll
  for (int t = 0; t < EPL; ++t) v[t] *= a.scale;
  const int64_t off = j * a.d + col;
  if (a.parts.rows) {
    float base[EPL];
#pragma unroll
    for (int t = 0; t < EPL; ++t) base[t] = 0.0f;
    a.parts.each(j, [&](int64_t at) {
      const float4* h = reinterpret_cast<const float4*>(a.parts.rows + at * a.d + col);
#pragma unroll
      for (int t = 0; t < EPL / 4; ++t) {
        const float4 w = h[t];
        base[4 * t] += w.x;
        base[4 * t + 1] += w.y;
        base[4 * t + 2] += w.z;
        base[4 * t + 3] += w.w;
      }
    });
#pragma unroll
    for (int t = 0; t < EPL; ++t) v[t] += base[t];
  }
  if (a.b16) {
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.dtable) + off);
#pragma unroll
    for (int t = 0; t < EPL / 2; ++t) o[t] = bf16_of(v[2 * t]) | (bf16_of(v[2 * t + 1]) << 16);
    return;
  }
  float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.dtable) + off);
#pragma unroll
  for (int t = 0; t < EPL / 4; ++t) {
    float4 w = float4{v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]};
    if (a.acc) {
      const float4 h = o[t];
      w = float4{h.x + w.x, h.y + w.y, h.z + w.z, h.w + w.w};
    }
    o[t] = w;
  }
}

template <int EPL>
__device__ __forceinline__ void put_partial(float* p, const float (&v)[EPL]) {
#pragma unroll
  for (int t = 0; t < EPL / 4; ++t)
    reinterpret_cast<float4*>(p)[t] = float4{v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]};
}

template <class E, int LPR>
__global__ __launch_bounds__(EMB_THREADS) void k_embed_pieces(EmbGrad a) {
  constexpr int EPL = Piece16<E>::EPL;
  constexpr int RPI = WAVE / LPR;
  constexpr int UNR = 8;
  const int l = lane_id(), q = l / LPR;
  const int col = ((int)blockIdx.y * LPR + l % LPR) * EPL;
  const int64_t piece = ((int64_t)blockIdx.x * (EMB_THREADS / WAVE) + (threadIdx.x >> 6)) * RPI + q;
  const int64_t n = (int64_t)*a.ntot, t0 = piece * EMB_PIECE;
  if (t0 >= n || col >= a.d) return;
  const int64_t t1 = min(n, t0 + EMB_PIECE);
  const int prev = t0 > 0 ? a.K[t0 - 1] : -1, next = t1 < n ? a.K[t1] : -1;
  const E* __restrict__ dout = static_cast<const E*>(a.dout);
  int cur = -1;
  int64_t start = t0;
  float sum[EPL];
  auto flush = [&](int64_t end) {
    const bool head = start == t0 && cur == prev, tail = end == t1 && cur == next;
    if (!head && !tail)
      put_row<EPL>(a, cur, col, sum);
    else
      put_partial<EPL>(a.partial + (piece * 2 + (head ? 0 : 1)) * a.d + col, sum);
  };
  for (int64_t tb = t0; tb < t1; tb += UNR) {
    int key[UNR];
    u32x4 raw[UNR];
    float wgt[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const int64_t t = min(tb + u, t1 - 1);
      const int64_t i = a.V[t] & 0x7FFFFFFF;
      key[u] = a.K[t];
      raw[u] = *reinterpret_cast<const u32x4*>(dout + i * a.d + col);
      wgt[u] = a.weight ? a.weight[i * a.wstride] : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      if (tb + u >= t1) break;
      float v[EPL];
      unpack16(raw[u], v);
      if (a.weight)
#pragma unroll
        for (int t = 0; t < EPL; ++t) v[t] *= wgt[u];
      if (key[u] != cur) {
        if (cur >= 0) flush(tb + u);
        cur = key[u];
        start = tb + u;
#pragma unroll
        for (int t = 0; t < EPL; ++t) sum[t] = v[t];
      } else {
#pragma unroll
        for (int t = 0; t < EPL; ++t) sum[t] += v[t];
      }
    }
  }
  flush(t1);
}

// One workgroup per piece: if a run starts in it and goes on, the run's partial rows
// are added, lane group g taking every (256 / LPR)-th of them, then the groups in order.
template <int LPR>
__global__ __launch_bounds__(EMB_THREADS) void k_embed_join(EmbGrad a) {
  constexpr int EPL = 8;
  constexpr int NG = EMB_THREADS / LPR;
  __shared__ float sh[NG][LPR * EPL + 4];
  const int64_t piece = blockIdx.x;
  const int64_t n = (int64_t)*a.ntot, t0 = piece * EMB_PIECE, t1 = t0 + EMB_PIECE;
  if (t1 >= n) return;
  const int j = a.K[t1 - 1];
  if (a.K[t1] != j || (t0 > 0 && a.K[t0] == j && a.K[t0 - 1] == j)) return;
  int64_t lo = t1, hi = n;   // first record beyond the run is in (lo, hi]
  while (hi - lo > 1) {
    const int64_t m = (lo + hi) / 2;
    if (a.K[m] == j) lo = m; else hi = m;
  }
  const int64_t last = lo / EMB_PIECE;
  const int g = threadIdx.x / LPR, sub = threadIdx.x % LPR;
  const int col = ((int)blockIdx.y * LPR + sub) * EPL;
  float sum[EPL];
#pragma unroll
  for (int t = 0; t < EPL; ++t) sum[t] = 0.0f;
  if (col < a.d) {
    for (int64_t p = piece + g; p <= last; p += NG) {
      const float4* h = reinterpret_cast<const float4*>(a.partial + (p * 2 + (p == piece ? 1 : 0)) * a.d + col);
#pragma unroll
      for (int t = 0; t < EPL / 4; ++t) {
        const float4 w = h[t];
        sum[4 * t] += w.x;
        sum[4 * t + 1] += w.y;
        sum[4 * t + 2] += w.z;
        sum[4 * t + 3] += w.w;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < EPL; ++t) sh[g][sub * EPL + t] = sum[t];
  __syncthreads();
  if (g != 0 || col >= a.d) return;
  const int used = (int)min((int64_t)NG, last - piece + 1);
  for (int o = 1; o < used; ++o)
#pragma unroll
    for (int t = 0; t < EPL; ++t) sum[t] += sh[o][sub * EPL + t];
  put_row<EPL>(a, j, col, sum);
}

// Lanes per row: the power of two that holds a row's 16-byte pieces, at most a wave
// (wider rows take several column blocks).
int lanes_per_row(int pieces) {
  int l = 1;
  while (l < pieces && l < WAVE) l *= 2;
  return l;
}

#define EMB_LPR(MACRO, lpr)        \
  switch (lpr) {                   \
    case 1: MACRO(1); break;       \
    case 2: MACRO(2); break;       \
    case 4: MACRO(4); break;       \
    case 8: MACRO(8); break;       \
    case 16: MACRO(16); break;     \
    case 32: MACRO(32); break;     \
    default: MACRO(64); break;     \
  }

unsigned ceil_div(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

template <class E>
hipError_t forward_t(int64_t n, int64_t C, int d, float scale, const void* table, const int32_t* ids, void* out,
                     hipStream_t st) {
  const int pieces = d / Piece16<E>::EPL, lpr = lanes_per_row(pieces);
  const int64_t rows = (int64_t)(EMB_THREADS / lpr) * 4;   // per workgroup
  const dim3 grid(ceil_div(n, rows), ceil_div(pieces, lpr));
#define EMB_FWD(L)                                                                                                  \
  hipLaunchKernelGGL((k_embed_rows<E, L>), grid, dim3(EMB_THREADS), 0, st, static_cast<const E*>(table), ids, \
                     static_cast<E*>(out), n, C, d, scale)
  EMB_LPR(EMB_FWD, lpr)
#undef EMB_FWD
  return hipGetLastError();
}

template <class E>
hipError_t pieces_t(const EmbGrad& a, int64_t npieces, hipStream_t st) {
  const int pieces = a.d / Piece16<E>::EPL, lpr = lanes_per_row(pieces);
  const dim3 grid(ceil_div(npieces, EMB_THREADS / lpr), ceil_div(pieces, lpr));
#define EMB_PCS(L) hipLaunchKernelGGL((k_embed_pieces<E, L>), grid, dim3(EMB_THREADS), 0, st, a)
  EMB_LPR(EMB_PCS, lpr)
#undef EMB_PCS
  return hipGetLastError();
}

hipError_t join(const EmbGrad& a, int64_t npieces, hipStream_t st) {
  const int pieces = a.d / 8, lpr = lanes_per_row(pieces);
  const dim3 grid((unsigned)npieces, ceil_div(pieces, lpr));
#define EMB_JOIN(L) hipLaunchKernelGGL((k_embed_join<L>), grid, dim3(EMB_THREADS), 0, st, a)
  EMB_LPR(EMB_JOIN, lpr)
#undef EMB_JOIN
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

int64_t piece_count(int64_t n) { return (n + EMB_PIECE - 1) / EMB_PIECE; }

}  // namespace

size_t row_sums_bytes(int64_t n, int64_t C, int d) {
  if (n == 0) return 16;
  return align256(pair_sort_geom(n, C).scratch_bytes) + 4 * align256((size_t)n * 4) +
         align256((size_t)piece_count(n) * 2 * d * 4);
}

size_t embed_workspace_bytes(int64_t n, int64_t C, int d) { return row_sums_bytes(n, C, d); }

hipError_t embed_forward(bool bf16v, int64_t n, int64_t C, int d, float scale, const void* table, const int32_t* ids,
                         void* out, hipStream_t st) {
  return bf16v ? forward_t<bf16>(n, C, d, scale, table, ids, out, st)
               : forward_t<float>(n, C, d, scale, table, ids, out, st);
}

hipError_t embed_backward(bool bf16v, int64_t n, int64_t C, int d, float scale, bool grad_bf16, bool accumulate,
                          const int32_t* ids, const void* dout, void* ws, void* dtable, hipStream_t st) {
  if (!accumulate) {
    const int64_t n16 = C * d * (grad_bf16 ? 2 : 4) / 16;
    const int64_t blocks = std::min<int64_t>((n16 + EMB_THREADS - 1) / EMB_THREADS, 4096);
    hipLaunchKernelGGL(k_embed_clear, dim3((unsigned)blocks), dim3(EMB_THREADS), 0, st, static_cast<u32x4*>(dtable), n16);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  RowSums r{};
  r.bf16v = bf16v;
  r.n = n;
  r.C = C;
  r.d = d;
  r.scale = scale;
  r.grad_bf16 = grad_bf16;
  r.accumulate = accumulate;
  r.ids = ids;
  r.rows = dout;
  return row_sums(r, ws, dtable, st);
}

hipError_t row_sums(const RowSums& r, void* ws, void* out, hipStream_t st) {
  const int64_t n = r.n;
  if (n == 0) return hipSuccess;
  const PairSortGeom g = pair_sort_geom(n, r.C);
  char* p = static_cast<char*>(ws);
  void* scratch = p;
  p += align256(g.scratch_bytes);
  int32_t* buf[4];
  for (int q = 0; q < 4; ++q, p += align256((size_t)n * 4)) buf[q] = reinterpret_cast<int32_t*>(p);
  EmbGrad a{};
  // no list entries: the records are the positions' ids alone
  hipError_t e = launch_pair_sort(g, r.ids, 0, 1, n, r.ids, r.C, scratch, buf[0], buf[1], buf[2], buf[3], &a.K, &a.V, &a.ntot, st);
  if (e != hipSuccess) return e;
  a.dout = r.rows;
  a.weight = r.weight;
  a.wstride = r.wstride;
  if (r.parts) a.parts = *r.parts;
  a.partial = reinterpret_cast<float*>(p);
  a.dtable = out;
  a.d = r.d;
  a.scale = r.scale;
  a.b16 = r.grad_bf16;
  a.acc = r.accumulate;
  const int64_t np = piece_count(n);
  e = r.bf16v ? pieces_t<bf16>(a, np, st) : pieces_t<float>(a, np, st);
  if (e != hipSuccess) return e;
  return join(a, np, st);
}

}  // namespace rece
