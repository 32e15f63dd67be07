// Item embedding: rows of the item table as a model's inputs, and the table's gradient.
//   forward   out_i = scale * table[ids_i]  (padding ids: zero rows)
//   backward  dtable_j = scale * sum over i with ids_i = j of dout_i
// Both are bound by memory.  Rows move as 16-byte pieces: LPR lanes (a power of two)
// per row, 64 / LPR rows per wave instruction, several rows in flight per lane group.
// The backward pass sorts (id, i) by id (stable), cuts the sorted records into fixed
// pieces and sums each piece's runs in float32 registers; a run inside one piece is
// written at once, a run over several pieces leaves one partial row per piece that a
// second kernel adds in a fixed order, so every result is reproducible bit for bit.
// Measured (MI355X, bf16 rows, float32 gradient):
//   256 rows of 64 floats            call 7.4 us (kernel 3.1 us: the call's own time bounds it)
//   51,200 rows of 64, 30,000 items  forward 5.2 us (13 MB), backward 34 us: sort 24, pieces 5, joins 7; latencies
//                                    of short launches, 27 MB in all
//   25,600 rows of 128, 1M items     forward and backward 113 us, 525 MB (512 MB of it the cleared gradient): 4.6 TB/s;
//                                    with a bf16 gradient 64 us, adding to a float32 one 38 us
#include <algorithm>

#include "rece_device.h"
#include "rece_ops.h"

namespace rece {

namespace {

constexpr int EMB_THREADS = 256;
constexpr int ORD_THREADS = 1024;
constexpr int ORD_TILE = 4096;      // records per workgroup of the sort
constexpr int ORD_BITS = 10;        // largest digit
constexpr int ORD_BINS = 1 << ORD_BITS;
constexpr int64_t ORD_TILES = 64;   // beyond these the library's longer sort, with a scan of its own, takes over
constexpr int EMB_PIECE = 8;        // sorted records per piece (51,200 records: 8 a piece 6.5 us, 32 a piece 12 us)

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
// Share `part` of `parts` of a region cleared by the `n` workgroups given (1024 threads each).
struct ClearArgs {
  u32x4* p;
  int64_t n16;   // 16-byte pieces of the region
};
__device__ __forceinline__ void clear_share(const ClearArgs& c, int part, int parts, int64_t b, int64_t n) {
  const int64_t lo = c.n16 * part / parts, hi = c.n16 * (part + 1) / parts;
  constexpr int UNR = 4;
  for (int64_t t = lo + b * (ORD_THREADS * UNR) + threadIdx.x; t < hi; t += n * (ORD_THREADS * UNR))
#pragma unroll
    for (int u = 0; u < UNR; ++u)
      if (t + u * ORD_THREADS < hi) __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, c.p + t + u * ORD_THREADS);
}

__global__ __launch_bounds__(ORD_THREADS) void k_embed_clear(ClearArgs c) { clear_share(c, 0, 1, blockIdx.x, gridDim.x); }

// ------------------------------------------------------------------ rows in the order of their ids
// Stable counting sort of the records (id, row) by digits of up to 10 bits, over tiles of 1024 to 4096 records.
//   k_order_hist     per tile, the count of every value of a digit;
//   k_order_scatter  per tile: every workgroup forms the digits' starting slots from all tiles' counts by
//                    itself (at most 64 tiles: 256 KB that lie in the L2; a scan of its own would be three
//                    more launches of a few us each), ranks its records in input order and writes them out.
// Integer atomics in LDS only, so the order is the same on every run.  Further workgroups of these launches
// clear the gradient meanwhile (the sort is latency, the clearing bandwidth).
struct OrderArgs {
  const int32_t* ids;      // first pass
  const int32_t *kin, *vin;
  int32_t *kout, *vout;
  int64_t n, C;
  int tiles, shift, bits;
  uint32_t* counts;        // [tiles][ORD_BINS] of this digit
  uint32_t* ntot;
  ClearArgs clear;
  int part, parts;
};

// Record t of a pass (id -1: none).
template <bool FIRST>
__device__ __forceinline__ int order_key(const OrderArgs& a, int64_t t, int64_t n) {
  if (t >= n) return -1;
  if constexpr (!FIRST) return a.kin[t];
  const int k = a.ids[t];
  return k < a.C ? k : -1;
}

template <bool FIRST, int PER>
__global__ __launch_bounds__(ORD_THREADS) void k_order_hist(OrderArgs a) {
  __shared__ uint32_t hist[ORD_BINS];
  const int tid = threadIdx.x, tile = blockIdx.x;
  if (tile >= a.tiles) {
    clear_share(a.clear, a.part, a.parts, tile - a.tiles, (int64_t)gridDim.x - a.tiles);
    return;
  }
  const int64_t n = FIRST ? a.n : (int64_t)*a.ntot;
  hist[tid] = 0u;
  int key[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) key[u] = order_key<FIRST>(a, (int64_t)tile * (PER * ORD_THREADS) + u * ORD_THREADS + tid, n);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    // one add for a wave of equal digits (popular ids after the first pass); others one by one
    const int dig = key[u] >= 0 ? (int)((uint32_t)key[u] >> a.shift & ((1u << a.bits) - 1u)) : -1;
    const int first = __builtin_amdgcn_readfirstlane(dig);
    if (ballot(dig == first) == ~0ull) {
      if (lane_id() == 0 && first >= 0) atomicAdd(&hist[first], (uint32_t)WAVE);
    } else if (dig >= 0) {
      atomicAdd(&hist[dig], 1u);
    }
  }
  __syncthreads();
  a.counts[(int64_t)tile * ORD_BINS + tid] = hist[tid];
}

// Exclusive prefix over the workgroup's threads (sh: one word per wave).
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* sh, uint32_t* total) {
  const int w = threadIdx.x / WAVE;
  const uint32_t incl = wave_prefix_incl(v);
  __syncthreads();
  if (lane_id() == WAVE - 1) sh[w] = incl;
  __syncthreads();
  uint32_t pre = 0, tot = 0;
#pragma unroll
  for (int q = 0; q < ORD_THREADS / WAVE; ++q) {
    if (q < w) pre += sh[q];
    tot += sh[q];
  }
  *total = tot;
  return pre + incl - v;
}

// Ranks PER x 64 consecutive records per wave among the tile's records with the same digit: cnt[wave][digit]
// becomes the number in earlier waves, at[q] the number in the wave before record q.
template <int PER>
__device__ __forceinline__ void order_rank(uint16_t (*cnt)[ORD_BINS], const int (&dig)[PER], int bits, uint32_t (&at)[PER],
                                           uint32_t* tot) {
  const int tid = threadIdx.x, w = tid / WAVE;
#pragma unroll
  for (int q = 0; q < ORD_THREADS / WAVE; ++q) cnt[q][tid] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const bool on = dig[q] >= 0;
    uint64_t same = ballot(on);
    for (int bit = 0; bit < bits; ++bit) {
      const bool one = (dig[q] >> bit) & 1;
      const uint64_t m = ballot(one);
      same &= one ? m : ~m;
    }
    const uint32_t rank = popc(same & lanemask_lt());
    const uint32_t base = on ? cnt[w][dig[q]] : 0u;
    wave_sync();
    if (on && rank == 0) cnt[w][dig[q]] = (uint16_t)(base + popc(same));
    wave_sync();
    at[q] = base + rank;
  }
  __syncthreads();
  uint32_t run = 0;
#pragma unroll
  for (int q = 0; q < ORD_THREADS / WAVE; ++q) {
    const uint32_t c = cnt[q][tid];
    cnt[q][tid] = (uint16_t)run;
    run += c;
  }
  *tot = run;   // of digit tid
}

template <bool FIRST, int PER>
__global__ __launch_bounds__(ORD_THREADS) void k_order_scatter(OrderArgs a) {
  __shared__ uint16_t cnt[ORD_THREADS / WAVE][ORD_BINS];
  __shared__ uint32_t start[ORD_BINS];
  __shared__ uint32_t sh[ORD_THREADS / WAVE];
  const int tid = threadIdx.x, w = tid / WAVE, l = lane_id(), tile = blockIdx.x;
  if (tile >= a.tiles) {
    clear_share(a.clear, a.part, a.parts, tile - a.tiles, (int64_t)gridDim.x - a.tiles);
    return;
  }
  const int64_t n = FIRST ? a.n : (int64_t)*a.ntot;
  int key[PER], val[PER], dig[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int64_t t = (int64_t)tile * (PER * ORD_THREADS) + (w * PER + q) * WAVE + l;
    key[q] = order_key<FIRST>(a, t, n);
    val[q] = FIRST ? (int)t : (t < n ? a.vin[t] : 0);
  }
  uint32_t before = 0, all = 0;   // records of digit tid: in earlier tiles, in all
#pragma unroll 8
  for (int t = 0; t < a.tiles; ++t) {
    const uint32_t c = a.counts[(int64_t)t * ORD_BINS + tid];
    before += t < tile ? c : 0u;
    all += c;
  }
#pragma unroll
  for (int q = 0; q < PER; ++q)
    dig[q] = key[q] >= 0 ? (int)((uint32_t)key[q] >> a.shift & ((1u << a.bits) - 1u)) : -1;
  uint32_t total, at[PER], in_tile;
  start[tid] = block_prefix(all, sh, &total) + before;
  if (FIRST && tile == 0 && tid == 0) *a.ntot = total;
  order_rank(cnt, dig, a.bits, at, &in_tile);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (dig[q] < 0) continue;
    const uint32_t slot = start[dig[q]] + cnt[w][dig[q]] + at[q];
    a.kout[slot] = key[q];
    a.vout[slot] = val[q];
  }
}

// Up to one tile: all digits in one workgroup, the records between passes in LDS.
__global__ __launch_bounds__(ORD_THREADS) void k_order_small(OrderArgs a, int key_bits) {
  __shared__ uint16_t cnt[ORD_THREADS / WAVE][ORD_BINS];
  __shared__ uint32_t start[ORD_BINS];
  __shared__ uint32_t sh[ORD_THREADS / WAVE];
  __shared__ int32_t sk[ORD_TILE], sv[ORD_TILE];
  const int tid = threadIdx.x, w = tid / WAVE, l = lane_id();
  if (blockIdx.x > 0) {
    clear_share(a.clear, 0, 1, (int64_t)blockIdx.x - 1, (int64_t)gridDim.x - 1);
    return;
  }
  int key[4], val[4], dig[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int t = (w * 4 + q) * WAVE + l;
    key[q] = order_key<true>(a, t, a.n);
    val[q] = t;
  }
  uint32_t total = 0;
  for (int shift = 0;;) {
    const int passes = (key_bits - shift + ORD_BITS - 1) / ORD_BITS, bits = (key_bits - shift + passes - 1) / passes;
#pragma unroll
    for (int q = 0; q < 4; ++q) dig[q] = key[q] >= 0 ? (int)((uint32_t)key[q] >> shift & ((1u << bits) - 1u)) : -1;
    uint32_t at[4], in_tile;
    order_rank(cnt, dig, bits, at, &in_tile);
    start[tid] = block_prefix(in_tile, sh, &total);
    __syncthreads();
    shift += bits;
    const bool last = shift >= key_bits;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (dig[q] < 0) continue;
      const uint32_t slot = start[dig[q]] + cnt[w][dig[q]] + at[q];
      if (last) {
        a.kout[slot] = key[q];
        a.vout[slot] = val[q];
      } else {
        sk[slot] = key[q];
        sv[slot] = val[q];
      }
    }
    if (last) break;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t t = (w * 4 + q) * WAVE + l;
      key[q] = t < total ? sk[t] : -1;
      val[q] = t < total ? sv[t] : 0;
    }
    __syncthreads();
  }
  if (tid == 0) *a.ntot = total;
}

struct EmbGrad {
  const int32_t* K;        // sorted ids
  const int32_t* V;        // their rows (bit 31 may be set)
  const uint32_t* ntot;    // records
  const void* dout;
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
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const int64_t t = min(tb + u, t1 - 1);
      const int64_t i = a.V[t] & 0x7FFFFFFF;
      key[u] = a.K[t];
      raw[u] = *reinterpret_cast<const u32x4*>(dout + i * a.d + col);
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      if (tb + u >= t1) break;
      float v[EPL];
      unpack16(raw[u], v);
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
  const int64_t piece = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  const int64_t n = (int64_t)*a.ntot, t0 = piece * EMB_PIECE, t1 = t0 + EMB_PIECE;
  if (t1 >= n) return;
  const int j = a.K[t1 - 1];
  if (a.K[t1] != j || (t0 > 0 && a.K[t0] == j && a.K[t0 - 1] == j)) return;
  int64_t lo = t1, hi = n;   // first record beyond the run is in (lo, hi]; a wave probes 64 places at a time
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + WAVE) / (WAVE + 1), m = lo + step * (lane_id() + 1);
    const int hits = popc(ballot(m < hi && a.K[m < hi ? m : lo] == j));   // sorted: the first lanes
    hi = min(hi, lo + step * (hits + 1));
    lo += step * hits;
  }
  const int64_t last = lo / EMB_PIECE;
  const int g = threadIdx.x / LPR, sub = threadIdx.x % LPR;
  const int col = ((int)blockIdx.y * LPR + sub) * EPL;
  float sum[EPL];
#pragma unroll
  for (int t = 0; t < EPL; ++t) sum[t] = 0.0f;
  if (col < a.d) {
#pragma unroll 4
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
  const int64_t x = std::min<int64_t>(npieces, 1 << 22);   // at most 2^30 threads along x
  const dim3 grid((unsigned)x, ceil_div(pieces, lpr), ceil_div(npieces, x));
#define EMB_JOIN(L) hipLaunchKernelGGL((k_embed_join<L>), grid, dim3(EMB_THREADS), 0, st, a)
  EMB_LPR(EMB_JOIN, lpr)
#undef EMB_JOIN
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

int64_t piece_count(int64_t n) { return (n + EMB_PIECE - 1) / EMB_PIECE; }

}  // namespace

namespace {

int key_bits(int64_t C) {
  int b = 1;
  while (((int64_t)1 << b) < C) ++b;
  return b;
}
int order_passes(int64_t C) { return (key_bits(C) + ORD_BITS - 1) / ORD_BITS; }
// Records per thread of the sort's tiles: as few as 64 tiles allow, so that many CUs rank (51,200 records, both
// digits: one per thread 23 us, two 25, four 31).
int order_per(int64_t n) {
  if (n <= ORD_TILE) return ORD_TILE / ORD_THREADS;   // one workgroup
  return n <= ORD_TILES * ORD_THREADS ? 1 : n <= 2 * ORD_TILES * ORD_THREADS ? 2 : ORD_TILE / ORD_THREADS;
}
int64_t order_tiles(int64_t n) {
  const int64_t tile = (int64_t)order_per(n) * ORD_THREADS;
  return (n + tile - 1) / tile;
}

// Scratch of the sort: the count matrices and the number of records, or the library's pair sort's.
size_t order_bytes(int64_t n, int64_t C) {
  if (order_tiles(n) > ORD_TILES) return align256(pair_sort_geom(n, C).scratch_bytes);
  return align256((size_t)order_tiles(n) * ORD_BINS * 4 + 16);
}

hipError_t clear_only(const ClearArgs& c, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>((c.n16 + 4 * ORD_THREADS - 1) / (4 * ORD_THREADS), 65536);
  hipLaunchKernelGGL(k_embed_clear, dim3((unsigned)blocks), dim3(ORD_THREADS), 0, st, c);
  return hipGetLastError();
}

// ids -> (K, V, ntot): ids in [0, C) in ascending order with their rows, equal ids in the order of their rows.
hipError_t order_rows(const int32_t* ids, int64_t n, int64_t C, const ClearArgs& clear, void* scratch, int32_t* const (&buf)[4],
                      EmbGrad& g, hipStream_t st) {
  const int64_t tiles = order_tiles(n);
  if (tiles > ORD_TILES) {
    if (clear.n16 > 0) {
      const hipError_t e = clear_only(clear, st);
      if (e != hipSuccess) return e;
    }
    // no list entries: the records are the rows' ids alone
    return launch_pair_sort(pair_sort_geom(n, C), ids, 0, 1, n, ids, C, scratch, buf[0], buf[1], buf[2], buf[3], &g.K,
                            &g.V, &g.ntot, st);
  }
  const int kb = key_bits(C), passes = order_passes(C), per = order_per(n);
  uint32_t* counts = static_cast<uint32_t*>(scratch);
  OrderArgs a{};
  a.ids = ids;
  a.n = n;
  a.C = C;
  a.tiles = (int)tiles;
  a.counts = counts;
  a.ntot = counts + tiles * ORD_BINS;
  a.clear = clear;
  a.parts = 2 * passes;
  // workgroups that clear, per launch: one at least where there is anything to clear (a table of one short row is
  // less than a piece per launch)
  const int64_t launches = tiles == 1 ? 1 : a.parts, share = (clear.n16 + launches - 1) / launches;
  const int64_t extra = std::min<int64_t>((share + 4 * ORD_THREADS - 1) / (4 * ORD_THREADS), 16384);
  if (tiles == 1) {
    a.kout = buf[0];
    a.vout = buf[1];
    hipLaunchKernelGGL(k_order_small, dim3((unsigned)(1 + extra)), dim3(ORD_THREADS), 0, st, a, kb);
    g.K = buf[0];
    g.V = buf[1];
    g.ntot = a.ntot;
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(tiles + extra));
  int shift = 0;
  for (int p = 0; p < passes; ++p) {
    const int left = passes - p, bits = (kb - shift + left - 1) / left;
    a.shift = shift;
    a.bits = bits;
    a.kout = buf[2 * (p & 1)];
    a.vout = buf[2 * (p & 1) + 1];
    for (int half = 0; half < 2; ++half) {
      a.part = 2 * p + half;
#define ORD_KERNEL(P)                                                         \
  (half == 0 ? (p == 0 ? k_order_hist<true, P> : k_order_hist<false, P>)      \
             : (p == 0 ? k_order_scatter<true, P> : k_order_scatter<false, P>))
      auto kern = per == 1 ? ORD_KERNEL(1) : per == 2 ? ORD_KERNEL(2) : ORD_KERNEL(4);
#undef ORD_KERNEL
      hipLaunchKernelGGL(kern, grid, dim3(ORD_THREADS), 0, st, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    a.kin = a.kout;
    a.vin = a.vout;
    shift += bits;
  }
  g.K = a.kout;
  g.V = a.vout;
  g.ntot = a.ntot;
  return hipSuccess;
}

}  // namespace

size_t embed_workspace_bytes(int64_t n, int64_t C, int d) {
  if (n == 0) return 16;
  return order_bytes(n, C) + 4 * align256((size_t)n * 4) + align256((size_t)piece_count(n) * 2 * d * 4);
}

hipError_t embed_forward(bool bf16v, int64_t n, int64_t C, int d, float scale, const void* table, const int32_t* ids,
                         void* out, hipStream_t st) {
  return bf16v ? forward_t<bf16>(n, C, d, scale, table, ids, out, st)
               : forward_t<float>(n, C, d, scale, table, ids, out, st);
}

hipError_t embed_backward(bool bf16v, int64_t n, int64_t C, int d, float scale, bool grad_bf16, bool accumulate,
                          const int32_t* ids, const void* dout, void* ws, void* dtable, hipStream_t st) {
  ClearArgs clear{};
  if (!accumulate) clear = ClearArgs{static_cast<u32x4*>(dtable), C * d * (grad_bf16 ? 2 : 4) / 16};
  if (n == 0) return clear.n16 > 0 ? clear_only(clear, st) : hipSuccess;
  char* p = static_cast<char*>(ws);
  void* scratch = p;
  p += order_bytes(n, C);
  int32_t* buf[4];
  for (int q = 0; q < 4; ++q, p += align256((size_t)n * 4)) buf[q] = reinterpret_cast<int32_t*>(p);
  EmbGrad a{};
  hipError_t e = order_rows(ids, n, C, clear, scratch, buf, a, st);
  if (e != hipSuccess) return e;
  a.dout = dout;
  a.partial = reinterpret_cast<float*>(p);
  a.dtable = dtable;
  a.d = d;
  a.scale = scale;
  a.b16 = grad_bf16;
  a.acc = accumulate;
  const int64_t np = piece_count(n);
  e = bf16v ? pieces_t<bf16>(a, np, st) : pieces_t<float>(a, np, st);
  if (e != hipSuccess) return e;
  return join(a, np, st);
}

}  // namespace rece
