// Causal attention over packed sequences of different lengths, grouped heads, with a learned bias by
// buckets of the distance, and its gradients (formulas in include/rece.h).  No array of scores exists: the
// softmax runs over the keys with a running maximum and sum.
//
// Products are formed transposed: a block S^T of 32 keys x 32 queries leaves lane l with query l % 32
// and 16 keys, so a query's maximum and sum need one exchange between two lanes, its factors are one
// register, and the block is the operand of the second product as it stands (rece_tile.h).
//   k_attn      owners = queries (32 per wave, their rows in registers), keys and values through LDS
//   k_attn_dq   the same sweep again: dq, and the exact row sums D_i = sum_j p_ij dp_ij
//   k_attn_dkv  owners = keys (32 per wave), the queries of all heads of a group through LDS: dk, dv and
//               the bias's gradient
// Tiles pass through two LDS buffers, the next tile's loads in flight during the current tile's work.
//
// Sequences are found by the workgroups themselves: with tiles of T rows, sequence u owns the slots
// from floor(o_u / T) + u on.  That number grows by at least ceil(length / T) from one sequence to the next, so
// the slots are distinct, floor(n / T) + n_seq of them are enough, and no list of tiles is made.
//
// Scores and sums are float32.  bf16: scores carry the factor log2(e); p and ds enter the second products as two bf16 terms
// (off by 2^-16 of them), so that out and the gradients are off by their own rounding alone.  One term's errors are as large
// as the results' rounding (out off by 1.25, dk and dv by 1.4 times it) for a tenth less time: 16 x 1,021 k_attn 71 us, with
// two terms 80; k_attn_dkv 168, 189.  float32: scores stay in natural units and their difference to the maximum is scaled.
// D comes from the outputs with what their rounding left (k_attn keeps it; from the rounded outputs alone dq would be off
// by 1.4 times as much).  What rounding is still in it would be the bias gradient's error: k_attn_dq adds the sum of
// p (dp - D) over the row to it, which is 0 for the exact D, for k_attn_dkv.
// float32: D keeps what the outputs' sums rounded, which no other row averages out: dq is off by 3.0e-7 to 6.3e-7 relative,
// 1.1 to 1.6 times the errors of a float32 form that sums p dp (k_attn_dkv's D has the remainder and does not have it).
// What bounds it: the time of one block in one wave, a chain of LDS reads, products and exponentials that two to four waves
// per SIMD hide in part (two for k_attn_dkv in bf16 at 64 wide: dk and dv are 64 registers, the keys' and values' rows 32, the
// next tile 32, scores and dp 32; with fragments and offsets 236 to 256); with few long sequences the longest one's last
// tile.  Vector units are busy 20 to 39 %, matrix units 3 to 22 % at 32 and 64 wide (float32 40 to 49 %) and 25 to 38 % at
// 128.  Measured (bf16 unless said; k_attn, k_attn_dq, k_attn_dkv in us):
//   256 x 150 tokens, 2 heads of 32, bias, gradients           19, 23, 40 (39 MB of rows, 3.5 GFLOP: startup and latencies)
//   200 x 200, 4 heads of 64, bias, gradients                  41, 47, 77
//   2,000 x 20, 4 heads of 64, bias, gradients                 45, 54, 73 (a wave for a sequence)
//   the same and one sequence of 10,000                        341, 369, 533 (a wave for each of its tiles, see query_waves)
//   16 x 1,021, 8 heads on 2 of 64, bias, gradients            79, 93, 190 (80 GFLOP, 220 TFLOP/s); float32 332, 469, 779
//   1 x 4,000, 4 heads on 1 of 64, bias, gradients             86, 89, 126
//   8 x 2,000, 8 heads of 128, gradients                       201, 246, 464 (306 GFLOP, 336 TFLOP/s)
//   3 x 2,731, 16 heads on 4 of 128, forward                   205 (122 GFLOP, 600 TFLOP/s)
// k_last is bound by the cache's rows where there are many, by its chain of launches and loads where there are few:
//   2,048 x 500, 4 heads of 64, bias  196 us (1.05 GB at 5.3 TB/s);  1 x 65,536, 8 heads on 2 of 128  18 us and the join 5
//   (67 MB; 2.9 TB/s in all);  5 x 200, 2 heads of 32  7 us
#include <algorithm>
#include <cmath>

#include "rece_device.h"
#include "rece_ops.h"
#include "rece_tile.h"

namespace rece {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float NO_WEIGHT = 1e30f;     // log-sum-exp of a row without weight: exp(t - 1e30) = 0
constexpr size_t MAX_LDS = 160 * 1024; // of a workgroup
constexpr int LAST_SPLITS = 256;       // parts of a sequence at most
constexpr int CLEAN = 64;              // workgroups that clear rows of no sequence

struct AttnArgs {
  const char* q;              // rows of heads of d elements; strides between rows in bytes
  const char* k;
  const char* v;
  const char* dout;           // [n][hq][d]
  char* out;                  // [n][hq][d]
  char* dq;
  char* dk;
  char* dv;
  int64_t qs, ks, vs, dqs, dks, dvs;
  const int32_t* offs;        // [n_seq + 1]
  const float* bias;          // [n_bounds + 1][hq] or nullptr
  char* low;                  // bf16: [n][hq][d] what the rounding of out left, or nullptr
  float2* lse;                // [hq][n] log-sum-exp (value, what its rounding left), or nullptr
  float* delta;               // [hq][n] D
  float* part;                // [slots][n_bounds + 1][hq] partial bias gradients
  int64_t n;
  int n_seq, d, hq, hk, slots;
  int hp;                     // k_attn_dkv: heads whose tables of the bias are in LDS at a time
  float scale, c;             // c: the factor of a product, with log2(e) for bf16
  int nbounds, dlast;         // dlast: from this distance on there is one bucket
  int32_t bounds[RECE_MAX_BOUNDS + 1];
};

struct SeqTile {
  int64_t begin;   // first row of the sequence
  int len;         // its rows; 0: the slot has no tile
  int first;       // first row of the tile within the sequence
};

// The tile of a slot (see above).  Every wave finds it by itself, 256 probes at a time.  What is found lies inside the
// rows whatever the offsets hold.
__device__ __forceinline__ SeqTile find_tile(const int32_t* offs, int n_seq, int64_t n, int slot, int T) {
  int lo = 0, size = n_seq;
  const int l = lane_id();
  auto clamped = [&](int u) { return max(0, min(offs[u], (int32_t)n)); };
  SeqTile t{0, 0, 0};
  while (true) {
    const int step = (int)(((int64_t)size + 255) / 256);
    int cnt = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t d = (int64_t)(4 * l + x) * step;
      const int at = lo + (int)(d < size ? d : 0);
      cnt += popc(ballot(d < size && clamped(at) / T + at <= slot));
    }
    if (cnt == 0) return t;
    lo += (cnt - 1) * step;
    if (step == 1) break;
    size = min(step, size - (cnt - 1) * step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int b = clamped(lo), e = max(b, clamped(lo + 1));
  t.begin = __builtin_amdgcn_readfirstlane(b);
  t.first = __builtin_amdgcn_readfirstlane((slot - (b / T + lo)) * T);
  t.len = __builtin_amdgcn_readfirstlane(t.first < e - b && t.first >= 0 ? e - b : 0);
  return t;
}

// Rows before the first and behind the last sequence become zero.
__device__ __forceinline__ void clean_rows(const AttnArgs& a, int which, int nt, char* p, int64_t stride, int row_bytes) {
  const int64_t first = max(0, min(a.offs[0], (int32_t)a.n)), last = max(first, (int64_t)min(a.offs[a.n_seq], (int32_t)a.n));
  const int cpr = row_bytes / 16;
  const int64_t rows = first + (a.n - last);
  for (int64_t t = (int64_t)which * nt + threadIdx.x; t < rows * cpr; t += (int64_t)CLEAN * nt) {
    const int64_t r = t / cpr, row = r < first ? r : last + (r - first);
    *reinterpret_cast<u32x4*>(p + row * stride + t % cpr * 16) = u32x4{0u, 0u, 0u, 0u};
  }
}

// TI rows of D elements from memory to LDS by NT threads (a workgroup or a wave), PT chunks each.  Rows beyond the end
// repeat the sequence's last one, whose weights there are 0.  Threads of chunks beyond the head copy its last one once more:
// those chunks stay 0 in LDS (the owners' elements there are 0 too, but 0 times an infinity would be NaN).  Whole tiles
// take one lane offset beside scalar ones.
template <class E, int D, int NT, int TI> struct Copy {
  using T = TileRows<E, D>;
  static constexpr int PT = TI * T::CPR / NT, BYTES = TI * T::RB;
  static constexpr int RPQ = NT / T::CPR;                   // rows of a step
  static constexpr int NV = RPQ >= 8 ? 1 : 8 / RPQ;         // the swizzle repeats every 8 rows
  static_assert(TI * T::CPR % NT == 0 && NT % T::CPR == 0, "whole chunks per thread, whole rows per step");
  u32x4 r[PT];
  uint32_t off, to[NV];
  static __device__ __forceinline__ uint32_t place(int row, int c) { return row * T::RB + ((c ^ (row & T::SWM)) << 4); }
  __device__ __forceinline__ void init(int64_t stride, int cpr) {
    const int i = (int)threadIdx.x % NT, row = i / T::CPR, c = min(i % T::CPR, cpr - 1);
    off = (uint32_t)row * (uint32_t)stride + c * 16;
#pragma unroll
    for (int v = 0; v < NV; ++v) to[v] = place(row + v * RPQ, c) - v * RPQ * T::RB;
  }
  // chunks beyond the head, once for each buffer
  static __device__ __forceinline__ void clear(uint32_t buf, int cpr) {
    const int i = (int)threadIdx.x % NT;
    if (i % T::CPR >= cpr)
      for (int q = 0; q < PT; ++q) lds_put(buf + place(i / T::CPR + q * RPQ, i % T::CPR), u32x4{0u, 0u, 0u, 0u});
  }
  __device__ __forceinline__ void fetch(const char* head, int64_t stride, int row0, int len) {
    const char* p = head + row0 * stride;
    if (row0 + TI <= len) {
#pragma unroll
      for (int q = 0; q < PT; ++q) r[q] = *reinterpret_cast<const u32x4*>(p + q * RPQ * stride + off);
    } else {
      const int row = (int)threadIdx.x % NT / T::CPR;
#pragma unroll
      for (int q = 0; q < PT; ++q)   // rows back to the last one
        r[q] = *reinterpret_cast<const u32x4*>(p + (q * RPQ - max(0, row0 + q * RPQ + row - (len - 1))) * stride + off);
    }
  }
  __device__ __forceinline__ void stash(uint32_t buf) const {
#pragma unroll
    for (int q = 0; q < PT; ++q) lds_put(buf + to[q % NV] + q * RPQ * T::RB, r[q]);
  }
};

// A wave's 32 rows as an operand: chunks 2 k + h of row l % 32.
template <class E, int D> struct Owners {
  static constexpr int KC = TileRows<E, D>::RB / 32;
  u32x4 v[KC];
  __device__ __forceinline__ void load(const char* head, int64_t stride, int row0, int len, int cpr) {
    const int l = lane_id(), h = l >> 5, row = row0 + (l & 31);
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      v[k] = u32x4{0u, 0u, 0u, 0u};
      if (row < len && 2 * k + h < cpr) v[k] = *reinterpret_cast<const u32x4*>(head + row * stride + (2 * k + h) * 16);
    }
  }
};

// The values are taken as loaded here: reads issued together are waited for once (left to itself the compiler waits for
// each read before its product and issues the next one after it).
template <class V, int N>
__device__ __forceinline__ void together(V (&f)[N]) {
#pragma unroll
  for (int q = 0; q < N; ++q) asm volatile("" : "+v"(f[q]));
}

// block[32 rows of the tile at base][32 owners], reads in batches of up to 8 fragments
template <class E, int D>
__device__ __forceinline__ f32x16 block_of(const TileReads<E, D>& o, uint32_t base, const Owners<E, D>& own) {
  constexpr int KC = Owners<E, D>::KC, B = KC < 8 ? KC : 8;
  f32x16 s = {};
#pragma unroll
  for (int k0 = 0; k0 < KC; k0 += B) {
    u32x4 f[B];
#pragma unroll
    for (int k = 0; k < B; ++k) f[k] = TileReads<E, D>::frag(o, base, k0 + k);
    together(f);
#pragma unroll
    for (int k = 0; k < B; ++k) s = TileMma<E>::run(f[k], own.v[k0 + k], s);
  }
  return s;
}

// acc[nb][32 coordinates][32 owners] += rows^T[coordinates][32 rows] g[32 rows][32 owners].  bf16: g rounded to bf16
// and the rounding of what that left, off by 2^-16 of g.  The second term takes the first one's registers: formed side by
// side they cost k_attn_dq at 64 wide its third wave per SIMD (200 x 200: 48 and 59 us).
template <class E, int D>
__device__ __forceinline__ void add_product(f32x16 (&acc)[D / 32], const f32x16& g, const TileReads<E, D>& o, uint32_t base) {
  if constexpr (sizeof(E) == 2) {
    constexpr int N = D / 32;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4 b, f[N];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = pack_bf16(g[8 * kk + 2 * e], g[8 * kk + 2 * e + 1]);
#pragma unroll
      for (int nb = 0; nb < N; ++nb) f[nb] = TileReads<E, D>::across(o, base, nb, kk);
      together(f);
#pragma unroll
      for (int nb = 0; nb < N; ++nb) acc[nb] = TileMma<E>::run(f[nb], b, acc[nb]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[e] = pack_bf16(g[8 * kk + 2 * e] - lo_f32(b[e]), g[8 * kk + 2 * e + 1] - hi_f32(b[e]));
#pragma unroll
      for (int nb = 0; nb < N; ++nb) acc[nb] = TileMma<E>::run(f[nb], b, acc[nb]);
    }
  } else {
    constexpr int N = D / 32;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[4 * N];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int nb = 0; nb < N; ++nb) f[e * N + nb] = TileReads<E, D>::across1(o, base, nb, 4 * q + e);
      together(f);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int nb = 0; nb < N; ++nb) acc[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(f[e * N + nb], g[4 * q + e], acc[nb], 0, 0, 0);
    }
  }
}

// Rows of results: coordinates 32 nb + tile_row(v) + 4 h of owner l % 32.
template <class E, int D>
__device__ __forceinline__ void store_rows(char* head, int64_t stride, int row0, int len, int d, const f32x16 (&acc)[D / 32],
                                           float f) {
  const int l = lane_id(), h = l >> 5, row = row0 + (l & 31);
  if (row >= len) return;
  char* p = head + row * stride;
#pragma unroll
  for (int nb = 0; nb < D / 32; ++nb)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = 32 * nb + 8 * g + 4 * h;
      if (at < d) {
        if constexpr (sizeof(E) == 2)
          *reinterpret_cast<uint2*>(p + at * 2) = make_uint2(pack_bf16(acc[nb][4 * g] * f, acc[nb][4 * g + 1] * f),
                                                             pack_bf16(acc[nb][4 * g + 2] * f, acc[nb][4 * g + 3] * f));
        else
          *reinterpret_cast<f32x4*>(p + at * 4) =
              f32x4{acc[nb][4 * g] * f, acc[nb][4 * g + 1] * f, acc[nb][4 * g + 2] * f, acc[nb][4 * g + 3] * f};
      }
    }
}

// exp of a difference of scores, in the scores' unit (bf16: base 2)
template <class E>
__device__ __forceinline__ float exp_of(float t) {
  return __builtin_amdgcn_exp2f(sizeof(E) == 2 ? t : t * LOG2E);
}

// The bias by distance in LDS, in the scores' unit: words 0 .. dlast + 95.  Ascending: distance word - 32;
// else distance dlast + 63 - word.  Distances below 0 (masked) hold 0, those of at least dlast the last bucket's.
// A bias of at most -1e30 leaves no weight.
template <class E, bool ASC>
__device__ __forceinline__ void fill_bias(const AttnArgs& a, uint32_t lut, int head, int nt, int len) {
  // only distances that a sequence of this length has, up to a block's end, and the one that stands for all far ones
  const int reach = min(len + 31, a.dlast + 63);
  for (int u = threadIdx.x; u < reach + 34; u += nt) {
    const int dist = u == reach + 33 ? a.dlast + 63 : u - 32, t = ASC ? dist + 32 : a.dlast + 63 - dist;
    int bucket = 0;   // the bounds are the same for all lanes: a comparison each, and no search in memory
    for (int x = 0; x < a.nbounds; x += 8)
#pragma unroll
      for (int y = 0; y < 8; ++y) bucket += a.bounds[x + y] <= dist;   // behind the last one: no distance
    float b = dist < 0 ? 0.0f : a.bias[(int64_t)bucket * a.hq + head];
    b = b <= -NO_WEIGHT ? -__builtin_huge_valf() : sizeof(E) == 2 ? b * LOG2E : b;
    lds_put<float>(lut + 4 * t, b);
  }
}
__device__ __forceinline__ f32x4 lds_f4(uint32_t off) {   // four words at any word
  typedef f32x4 any __attribute__((aligned(4)));
  return *reinterpret_cast<const __attribute__((address_space(3))) any*>((uintptr_t)off);
}

// The products x of a block of 32 keys (rows, from j0) x 32 queries (from i0 >= j0), made ready: the scores are
// x mul + add, where `near` blocks have the bias in x already.
struct Affine {
  float mul, add;
};
template <class E, bool BIAS>
__device__ __forceinline__ Affine scores_keys(f32x16& x, float c, int i0, int j0, uint32_t lut, int dlast, float far) {
  const int l = lane_id(), h = l >> 5, r = l & 31;
  Affine f{c, far};
  if (BIAS && i0 - j0 - 31 < dlast) {
    const uint32_t at = lut + 4 * (dlast + 63 - (i0 - j0 + r - 4 * h));
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 b = lds_f4(at + 32 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * g + e] = fmaf(x[4 * g + e], c, b[e]);
    }
    f.mul = 1.0f;
    f.add = 0.0f;
  }
  if (j0 == i0) {
#pragma unroll
    for (int v = 0; v < 16; ++v) x[v] = tile_row(v) + 4 * h > r ? -__builtin_huge_valf() : x[v];
  }
  return f;
}

// Of k_attn and k_attn_dq: waves, their queries, and the keys of a tile.
template <class E, int DH, int NW> struct Shape {
  static constexpr int NT = 64 * NW;
  static constexpr int T = 32 * NW;
  static constexpr int TJ = NW == 1 || TileRows<E, DH>::RB > 256 ? 32 : 64;
  static constexpr int BYTES = TJ * TileRows<E, DH>::RB;
};

template <class E, int DH, int NW, bool BIAS>
__global__ __launch_bounds__(64 * NW, NW == 1 && sizeof(E) * DH > 256 ? 1 : 2) void k_attn(AttnArgs a) {
  using S = Shape<E, DH, NW>;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const uint32_t lut = lds0 + 4 * S::BYTES;
  const int es = sizeof(E), cpr = a.d * es / 16;
  const int64_t os = (int64_t)a.hq * a.d * es;
  const int b = blockIdx.x;
  if (b >= a.slots * a.hq) {
    clean_rows(a, b - a.slots * a.hq, S::NT, a.out, os, (int)os);
    return;
  }
  // last slots first: within a sequence they have the most keys
  const int head = b % a.hq, kvh = head / (a.hq / a.hk);
  const SeqTile st = find_tile(a.offs, a.n_seq, a.n, a.slots - 1 - b / a.hq, S::T);
  if (st.len == 0) return;
  const char* kh = a.k + st.begin * a.ks + (int64_t)kvh * a.d * es;
  const char* vh = a.v + st.begin * a.vs + (int64_t)kvh * a.d * es;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i0 = st.first + 32 * w;
  Owners<E, DH> q;
  q.load(a.q + st.begin * a.qs + (int64_t)head * a.d * es, a.qs, i0, st.len, cpr);
  TileReads<E, DH> o;
  o.init();
  f32x16 acc[DH / 32] = {};
  float m = NEG_INF, sum = 0.0f;
  const int nt = (min(st.first + S::T, st.len) + S::TJ - 1) / S::TJ;
  Copy<E, DH, S::NT, S::TJ> ck, cv;
  ck.init(a.ks, cpr);
  cv.init(a.vs, cpr);
  ck.fetch(kh, a.ks, 0, st.len);
  cv.fetch(vh, a.vs, 0, st.len);
  if constexpr (BIAS) fill_bias<E, false>(a, lut, head, S::NT, st.len);
  for (int x = 0; x < 4; ++x) ck.clear(lds0 + x * S::BYTES, cpr);
  ck.stash(lds0);
  cv.stash(lds0 + S::BYTES);
  __syncthreads();
  const float far = BIAS ? lds_at<float>(lut) : 0.0f;
  for (int t = 0; t < nt; ++t) {
    if (t + 1 < nt) {
      ck.fetch(kh, a.ks, (t + 1) * S::TJ, st.len);
      cv.fetch(vh, a.vs, (t + 1) * S::TJ, st.len);
    }
    const uint32_t kb = lds0 + (t & 1) * 2 * S::BYTES, vb = kb + S::BYTES;
#pragma unroll
    for (int jb = 0; jb < S::TJ / 32; ++jb) {
      const int j0 = t * S::TJ + 32 * jb;
      if (j0 > i0 || i0 >= st.len) continue;
      f32x16 x = block_of<E, DH>(o, kb + jb * 32 * TileRows<E, DH>::RB, q);
      const Affine af = scores_keys<E, BIAS>(x, a.c, i0, j0, lut, a.dlast, far);
      float bm = x[0];
#pragma unroll
      for (int v = 1; v < 16; ++v) bm = fmaxf(bm, x[v]);
      bm = fmaf(fmaxf(bm, __shfl_xor(bm, 32)), af.mul, af.add);
      // the reference follows the maximum in steps: terms stay below 2^8
      if (ballot(bm > m + (sizeof(E) == 2 ? 8.0f : 5.5f))) {
        const float up = fmaxf(m, bm);
        const float f = m == NEG_INF ? 0.0f : exp_of<E>(m - up);
        sum *= f;
#pragma unroll
        for (int nb = 0; nb < DH / 32; ++nb)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[nb][v] *= f;
        m = up;
      }
      const float off = af.add - fmaxf(m, -NO_WEIGHT);
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        x[v] = exp_of<E>(fmaf(x[v], af.mul, off));
        part[v & 1] += x[v];
      }
      sum += part[0] + part[1];
      add_product<E, DH>(acc, x, o, vb + jb * 32 * TileRows<E, DH>::RB);
    }
    if (t + 1 < nt) {
      const uint32_t nb = lds0 + ((t + 1) & 1) * 2 * S::BYTES;
      ck.stash(nb);
      cv.stash(nb + S::BYTES);
      __syncthreads();
    }
  }
  sum += __shfl_xor(sum, 32);
  store_rows<E, DH>(a.out + st.begin * os + (int64_t)head * a.d * es, os, i0, st.len, a.d, acc, sum == 0.0f ? 0.0f : 1.0f / sum);
  const int l = lane_id();
  if (sizeof(E) == 2 && a.low) {
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int nb = 0; nb < DH / 32; ++nb)
#pragma unroll
      for (int v = 0; v < 16; v += 2) {
        const float x = acc[nb][v] * f, y = acc[nb][v + 1] * f;
        const uint32_t p = pack_bf16(x, y);
        acc[nb][v] = x - lo_f32(p);
        acc[nb][v + 1] = y - hi_f32(p);
      }
    store_rows<E, DH>(a.low + st.begin * os + (int64_t)head * a.d * es, os, i0, st.len, a.d, acc, 1.0f);
  }
  if (a.lse && l < 32 && i0 + l < st.len) {
    float2 v = make_float2(NO_WEIGHT, 0.0f);
    if (sum != 0.0f) {
      const float lg = sizeof(E) == 2 ? log2f(sum) : logf(sum);
      v.x = m + lg;
      const float bb = v.x - m;
      v.y = (m - (v.x - bb)) + (lg - bb);
    }
    a.lse[(int64_t)head * a.n + st.begin + i0 + l] = v;
  }
}

template <class E, int DH, int NW, bool BIAS>
__global__ __launch_bounds__(64 * NW, sizeof(E) * DH <= (NW == 1 ? 128 : 256) ? 2 : 1) void k_attn_dq(AttnArgs a) {
  using S = Shape<E, DH, NW>;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const uint32_t lut = lds0 + 4 * S::BYTES;
  const int es = sizeof(E), cpr = a.d * es / 16;
  const int64_t os = (int64_t)a.hq * a.d * es;
  const int b = blockIdx.x;
  if (b >= a.slots * a.hq) {
    clean_rows(a, b - a.slots * a.hq, S::NT, a.dq, a.dqs, (int)os);
    return;
  }
  const int head = b % a.hq, kvh = head / (a.hq / a.hk);
  const SeqTile st = find_tile(a.offs, a.n_seq, a.n, a.slots - 1 - b / a.hq, S::T);
  if (st.len == 0) return;
  const int64_t hb = (int64_t)head * a.d * es;
  const char* kh = a.k + st.begin * a.ks + (int64_t)kvh * a.d * es;
  const char* vh = a.v + st.begin * a.vs + (int64_t)kvh * a.d * es;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l = lane_id();
  const int i0 = st.first + 32 * w;
  Owners<E, DH> q, go;
  q.load(a.q + st.begin * a.qs + hb, a.qs, i0, st.len, cpr);
  go.load(a.dout + st.begin * os + hb, os, i0, st.len, cpr);
  const bool live = i0 + (l & 31) < st.len;
  const int64_t row = (int64_t)head * a.n + st.begin + i0 + (l & 31);
  const float2 lse = live ? a.lse[row] : make_float2(NO_WEIGHT, 0.0f);
  float d0 = 0.0f;   // D by the outputs
#pragma unroll 1
  for (int part = 0; part < (int)(4 / sizeof(E)); ++part) {
    Owners<E, DH> ov;
    ov.load((part ? a.low : a.out) + st.begin * os + hb, os, i0, st.len, cpr);
#pragma unroll
    for (int k = 0; k < Owners<E, DH>::KC; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(E) == 2) {
          d0 = fmaf(lo_f32(ov.v[k][e]), lo_f32(go.v[k][e]), d0);
          d0 = fmaf(hi_f32(ov.v[k][e]), hi_f32(go.v[k][e]), d0);
        } else {
          d0 = fmaf(__uint_as_float(ov.v[k][e]), __uint_as_float(go.v[k][e]), d0);
        }
      }
  }
  d0 += __shfl_xor(d0, 32);
  TileReads<E, DH> o;
  o.init();
  f32x16 acc[DH / 32] = {};
  float rest = 0.0f;
  const int nt = (min(st.first + S::T, st.len) + S::TJ - 1) / S::TJ;
  Copy<E, DH, S::NT, S::TJ> ck, cv;
  ck.init(a.ks, cpr);
  cv.init(a.vs, cpr);
  ck.fetch(kh, a.ks, 0, st.len);
  cv.fetch(vh, a.vs, 0, st.len);
  if constexpr (BIAS) fill_bias<E, false>(a, lut, head, S::NT, st.len);
  for (int x = 0; x < 4; ++x) ck.clear(lds0 + x * S::BYTES, cpr);
  ck.stash(lds0);
  cv.stash(lds0 + S::BYTES);
  __syncthreads();
  const float far = BIAS ? lds_at<float>(lut) : 0.0f;
  for (int t = 0; t < nt; ++t) {
    if (t + 1 < nt) {
      ck.fetch(kh, a.ks, (t + 1) * S::TJ, st.len);
      cv.fetch(vh, a.vs, (t + 1) * S::TJ, st.len);
    }
    const uint32_t kb = lds0 + (t & 1) * 2 * S::BYTES, vb = kb + S::BYTES;
#pragma unroll
    for (int jb = 0; jb < S::TJ / 32; ++jb) {
      const int j0 = t * S::TJ + 32 * jb;
      if (j0 > i0 || i0 >= st.len) continue;
      const uint32_t at = jb * 32 * TileRows<E, DH>::RB;
      f32x16 x = block_of<E, DH>(o, kb + at, q);
      const f32x16 dp = block_of<E, DH>(o, vb + at, go);
      const Affine af = scores_keys<E, BIAS>(x, a.c, i0, j0, lut, a.dlast, far);
      const float off = sizeof(E) == 2 ? (af.add - lse.x) - lse.y : af.add - lse.x;   // (bf16: off by 2^-24 of it)
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        float s = fmaf(x[v], af.mul, off);
        if (sizeof(E) == 4) s -= lse.y;
        x[v] = exp_of<E>(s) * (dp[v] - d0);
        part[v & 1] += x[v];
      }
      rest += part[0] + part[1];
      add_product<E, DH>(acc, x, o, kb + at);
    }
    if (t + 1 < nt) {
      const uint32_t nb = lds0 + ((t + 1) & 1) * 2 * S::BYTES;
      ck.stash(nb);
      cv.stash(nb + S::BYTES);
      __syncthreads();
    }
  }
  rest += __shfl_xor(rest, 32);
  store_rows<E, DH>(a.dq + st.begin * a.dqs + hb, a.dqs, i0, st.len, a.d, acc, a.scale);
  if (l < 32 && live) a.delta[row] = d0 + rest;
}

constexpr int SKEW = 63 * 33 * 4;   // bytes of a block by distance

// One workgroup for 32 keys and a key head.  Its IW waves deal the group's (head, 32 queries) pairs among themselves, each
// with LDS of its own and no barrier on the way, and add up what they have at the end.  Where the tables of the bias of
// all heads of a group and its gradients do not fit in LDS, they take `hp` heads at a time.  Three waves per SIMD at 32 wide
// although a few registers go through memory (256 x 150 tokens: two waves 41.6, three 39.1 us).
template <class E, int DH, int IW, bool BIAS>
__global__ __launch_bounds__(64 * IW, sizeof(E) * DH <= 64 ? 3 : sizeof(E) * DH <= 128 ? 2 : 1) void k_attn_dkv(AttnArgs a) {
  constexpr int NT = 64 * IW, RB = TileRows<E, DH>::RB, BYTES = 32 * RB;
  constexpr bool AHEAD = RB <= 256;               // rows on the way during the work (wider ones do not fit in registers)
  constexpr bool REST = BIAS || sizeof(E) == 4;   // what the log-sum-exp's rounding left counts (dbias, float32)
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id(), h = l >> 5, r = l & 31;
  const uint32_t qb = lds0 + w * 2 * BYTES, gb = qb + BYTES;
  const uint32_t par = lds0 + IW * 2 * BYTES + w * 3 * 128;      // [3][32] log-sum-exp, its rest, D
  const int words = a.dlast + 96, hw = a.dlast + 34;
  const uint32_t lut0 = lds0 + IW * (2 * BYTES + 3 * 128);       // [hp][words] bias by distance
  const uint32_t hist0 = lut0 + 4 * words * a.hp;                // [IW][hp][hw] sums of ds by distance (word - 32), the last
                                                                 // word: of at least dlast
  const uint32_t skew = hist0 + 4 * hw * a.hp * IW + w * SKEW;   // [IW] blocks by distance
  const int es = sizeof(E), cpr = a.d * es / 16, group = a.hq / a.hk;
  const int64_t os = (int64_t)a.hq * a.d * es;
  const int b = blockIdx.x;
  if (b >= a.slots * a.hk) {
    const int which = b - a.slots * a.hk;
    clean_rows(a, which, NT, a.dk, a.dks, a.hk * a.d * es);
    clean_rows(a, which, NT, a.dv, a.dvs, a.hk * a.d * es);
    return;
  }
  const int kvh = b % a.hk, slot = b / a.hk, nbk = a.nbounds + 1;
  const SeqTile st = find_tile(a.offs, a.n_seq, a.n, slot, 32);
  if (st.len == 0) {
    if constexpr (BIAS)
      for (int t = tid; t < nbk * group; t += NT)
        a.part[((int64_t)slot * nbk + t / group) * a.hq + kvh * group + t % group] = 0.0f;
    return;
  }
  const int j0 = st.first, t0 = j0 / 32, nt = (st.len + 31) / 32 - t0;   // tiles of queries from t0 on
  Owners<E, DH> kk, vv;
  kk.load(a.k + st.begin * a.ks + (int64_t)kvh * a.d * es, a.ks, j0, st.len, cpr);
  vv.load(a.v + st.begin * a.vs + (int64_t)kvh * a.d * es, a.vs, j0, st.len, cpr);
  TileReads<E, DH> o;
  o.init();
  f32x16 dk[DH / 32] = {}, dv[DH / 32] = {};
  Copy<E, DH, 64, 32> cq, cg;
  cq.init(a.qs, cpr);
  cg.init(os, cpr);
  cq.clear(qb, cpr);
  cg.clear(gb, cpr);
  float2 nl = make_float2(0.0f, 0.0f);
  float nd = 0.0f;
  auto fetch = [&](int head, int t) {
    const int64_t hb = (int64_t)head * a.d * es;
    cq.fetch(a.q + st.begin * a.qs + hb, a.qs, t * 32, st.len);
    cg.fetch(a.dout + st.begin * os + hb, os, t * 32, st.len);
    const int i = t * 32 + r;
    const int64_t row = (int64_t)head * a.n + st.begin + i;
    nl = make_float2(NO_WEIGHT, 0.0f);
    nd = 0.0f;
    if (i < st.len) {
      nl = a.lse[row];
      nd = a.delta[row];
    }
  };
  if constexpr (BIAS)
    for (int t = l; t < SKEW / 4; t += 64) lds_put<float>(skew + 4 * t, 0.0f);
  for (int h0 = 0; h0 < group; h0 += a.hp) {
    const int nh = min(a.hp, group - h0), head0 = kvh * group + h0;
    int hh = w / nt, t = w - hh * nt;      // the wave's pair: a head of these, a tile
    if (AHEAD && hh < nh) fetch(head0 + hh, t0 + t);
    if constexpr (BIAS) {
      if (h0 > 0) __syncthreads();
      for (int x = 0; x < nh; ++x) fill_bias<E, true>(a, lut0 + 4 * words * x, head0 + x, NT, st.len);
      for (int x = l; x < nh * hw; x += 64) lds_put<float>(hist0 + 4 * (w * a.hp * hw + x), 0.0f);
      __syncthreads();
    }
    float far = 0.0f, farsum = 0.0f;       // of the head at hand: its far distances' bias, and their sum of ds
    int at_head = -1;
    uint32_t lut = lut0, hist = hist0;
    auto leave_head = [&]() {
      farsum = wave_sumf(farsum);
      if (l == 0 && at_head >= 0) lds_put<float>(hist + 4 * (hw - 1), farsum);
      farsum = 0.0f;
    };
    while (hh < nh) {
      if constexpr (BIAS) {
        if (hh != at_head) {
          leave_head();
          at_head = hh;
          lut = lut0 + 4 * words * hh;
          hist = hist0 + 4 * (w * a.hp + hh) * hw;
          far = lds_at<float>(lut + 4 * (words - 1));
        }
      }
      if (!AHEAD) fetch(head0 + hh, t0 + t);
      wave_sync();
      cq.stash(qb);
      cg.stash(gb);
      const int i0 = (t0 + t) * 32;
      const bool near = BIAS && i0 - j0 - 31 < a.dlast;
      if (h == 0) {
        lds_put<float>(par + 4 * r, nl.x);
        if (REST) lds_put<float>(par + 128 + 4 * r, near ? nl.y : nl.y - far);
        lds_put<float>(par + 256 + 4 * r, nd);
      }
      wave_sync();
      t += IW;
      while (t >= nt && hh < nh) {
        t -= nt;
        ++hh;
      }
      if (AHEAD && hh < nh) fetch(head0 + hh, t0 + t);
      f32x16 x = block_of<E, DH>(o, qb, kk);
      f32x16 dp = block_of<E, DH>(o, gb, vv);
      const uint32_t la = lut + 4 * (i0 - j0 - r + 4 * h + 32), pa = par + 16 * h;
      if (i0 == j0) {
#pragma unroll
        for (int v = 0; v < 16; ++v) x[v] = tile_row(v) + 4 * h < r ? NEG_INF : x[v];
      }
      if (near) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 bias = lds_f4(la + 32 * g), lh = lds_at<f32x4>(pa + 32 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * g + e] = fmaf(x[4 * g + e], a.c, bias[e]) - lh[e];
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 lh = lds_at<f32x4>(pa + 32 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * g + e] = fmaf(x[4 * g + e], a.c, -lh[e]);
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 ll = {0.0f, 0.0f, 0.0f, 0.0f};
        if (REST) ll = lds_at<f32x4>(pa + 128 + 32 * g);
        const f32x4 dd = lds_at<f32x4>(pa + 256 + 32 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = 4 * g + e;
          x[v] = exp_of<E>(REST ? x[v] - ll[e] : x[v]);
          dp[v] = x[v] * (dp[v] - dd[e]);
        }
        }
      add_product<E, DH>(dv, x, o, gb);
      add_product<E, DH>(dk, dp, o, qb);
      if constexpr (BIAS) {
        if (near) {
          // ds of query i and key j to word i of row i - j + 31 (33 words a row: lanes meet in no bank), what no pair has
          // stays 0; then lane x adds up row x
          const uint32_t at = skew + 4 * (33 * (4 * h - r + 31) + 4 * h);
#pragma unroll
          for (int v = 0; v < 16; ++v) lds_put<float>(at + 4 * 34 * tile_row(v), dp[v]);
          wave_sync();
          const uint32_t ha = hist + 4 * (i0 - j0 + 1 + l), ra = skew + 4 * 33 * min(l, 62);
          const bool in = i0 - j0 - 31 + l < a.dlast;
          float s[4] = {in ? lds_at<float>(ha) : farsum, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int y = 0; y < 32; ++y) s[y & 3] += lds_at<float>(ra + 4 * y);
          const float all = (s[0] + s[1]) + (s[2] + s[3]);
          if (l < 63) {
            if (in) lds_put<float>(ha, all);
            else farsum = all;
          }
        } else {
          float s[2] = {0.0f, 0.0f};
#pragma unroll
          for (int v = 0; v < 16; ++v) s[v & 1] += dp[v];
          farsum += s[0] + s[1];
        }
      }
    }
    if constexpr (BIAS) {
      leave_head();
      __syncthreads();
      // eight lanes to a bucket of a head
      for (int x = tid; x < ((nh * nbk * 8 + NT - 1) & ~(NT - 1)); x += NT) {
        const int k = x >> 3, hd = k / nbk, bk = k - hd * nbk;
        float s = 0.0f;
        if (hd < nh) {
          const uint32_t from = hist0 + 4 * hd * hw;
          if (bk == a.nbounds) {
            if ((x & 7) < IW) s = lds_at<float>(from + 4 * ((x & 7) * a.hp * hw + hw - 1));
          } else {
            for (int y = (bk == 0 ? 0 : a.bounds[bk - 1]) + (x & 7); y < a.bounds[bk]; y += 8)
#pragma unroll
              for (int q = 0; q < IW; ++q) s += lds_at<float>(from + 4 * (q * a.hp * hw + y + 32));
          }
        }
#pragma unroll
        for (int q = 4; q >= 1; q >>= 1) s += __shfl_xor(s, q);
        if (hd < nh && (x & 7) == 0) a.part[((int64_t)slot * nbk + bk) * a.hq + head0 + hd] = s;
      }
    }
  }
  if constexpr (IW == 1) {
    store_rows<E, DH>(a.dk + st.begin * a.dks + (int64_t)kvh * a.d * es, a.dks, j0, st.len, a.d, dk, a.scale);
    store_rows<E, DH>(a.dv + st.begin * a.dvs + (int64_t)kvh * a.d * es, a.dvs, j0, st.len, a.d, dv, 1.0f);
  } else {
    // [IW][32][DH] float32 through the tiles' LDS, 16-byte piece c of row q at c ^ (q & 7)
    auto join = [&](const f32x16 (&acc)[DH / 32], char* out, int64_t stride, float f) {
      __syncthreads();
#pragma unroll
      for (int nb = 0; nb < DH / 32; ++nb)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          lds_put(lds0 + (w * 32 + r) * DH * 4 + (((8 * nb + 2 * g + h) ^ (r & 7)) << 4),
                  f32x4{acc[nb][4 * g], acc[nb][4 * g + 1], acc[nb][4 * g + 2], acc[nb][4 * g + 3]});
      __syncthreads();
      constexpr int EPC = 16 / sizeof(E);          // elements of a 16-byte piece of the result
      for (int t = tid; t < 32 * (DH / EPC); t += NT) {
        const int row = t / (DH / EPC), c = t % (DH / EPC);
        if (j0 + row >= st.len || c >= cpr) continue;
        float y[EPC];
#pragma unroll
        for (int p = 0; p < EPC / 4; ++p) {
          f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < IW; ++q)
            s += lds_at<f32x4>(lds0 + (q * 32 + row) * DH * 4 + (((c * (EPC / 4) + p) ^ (row & 7)) << 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) y[4 * p + e] = s[e] * f;
        }
        u32x4 o4;
#pragma unroll
        for (int e = 0; e < 4; ++e) o4[e] = sizeof(E) == 2 ? pack_bf16(y[(2 * e) % EPC], y[(2 * e + 1) % EPC]) : __float_as_uint(y[e]);
        *reinterpret_cast<u32x4*>(out + (j0 + row) * stride + c * 16) = o4;
      }
    };
    join(dk, a.dk + st.begin * a.dks + (int64_t)kvh * a.d * es, a.dks, a.scale);
    join(dv, a.dv + st.begin * a.dvs + (int64_t)kvh * a.d * es, a.dvs, 1.0f);
  }
}

// ------------------------------------------------------------------ the last token of every sequence
struct LastArgs {
  const char* q;              // [n_seq] rows of hq heads
  const char* k;              // [rows] rows of hk heads
  const char* v;
  char* out;                  // [n_seq][hq][d]
  int64_t qs, ks, vs;
  const int32_t* begin;       // [n_seq]
  const int32_t* length;      // [n_seq]
  const float* bias;
  float* part;                // [n_seq][hq][splits][d] sums of p v, then [n_seq][hq][2][splits]: reference, sum of p
  int64_t rows;
  int n_seq, d, hq, hk, splits;
  float c;
  int nbounds, dlast;
  int32_t bounds[RECE_MAX_BOUNDS];
};

// One workgroup for a sequence, a key head and a part of the keys.  The query heads of the group are the columns
// of a block (up to 32), so keys and values are read once.  Every wave goes over blocks of 32 keys by itself, with LDS of
// its own; the four are joined at the end, and the parts of a sequence by k_last_join.
template <class E, int DH, bool BIAS>
__global__ __launch_bounds__(256, sizeof(E) * DH > 256 ? 1 : 2) void k_last(LastArgs a) {
  constexpr int RB = TileRows<E, DH>::RB, BYTES = 32 * RB, P = DH + 4;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const int group = a.hq / a.hk;
  const uint32_t map = lds0 + max(8 * BYTES, 16 * group * P);   // bucket of every distance up to dlast, a byte each
  const int es = sizeof(E), cpr = a.d * es / 16;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id(), h = l >> 5, r = l & 31;
  const int kvh = blockIdx.x % a.hk, u = blockIdx.x / a.hk % a.n_seq, split = blockIdx.x / a.hk / a.n_seq;
  const int64_t begin = min(max((int64_t)a.begin[u], (int64_t)0), a.rows);
  const int len = (int)min(max((int64_t)a.length[u], (int64_t)0), a.rows - begin);
  const int head = kvh * group + min(r, group - 1);
  Owners<E, DH> q;
  q.load(a.q + u * a.qs + (int64_t)kvh * group * a.d * es, (int64_t)a.d * es, 0, group, cpr);
  const char* kh = a.k + begin * a.ks + (int64_t)kvh * a.d * es;
  const char* vh = a.v + begin * a.vs + (int64_t)kvh * a.d * es;
  float far = 0.0f;
  auto unit = [](float b) { return b <= -NO_WEIGHT ? NEG_INF : sizeof(E) == 2 ? b * LOG2E : b; };
  if constexpr (BIAS) {
    for (int t = tid; t <= a.dlast; t += 256) {
      int lo = 0, hi = a.nbounds;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.bounds[mid] <= t) lo = mid + 1;
        else hi = mid;
      }
      lds_put<uint8_t>(map + t, (uint8_t)lo);
    }
    far = unit(a.bias[(int64_t)a.nbounds * a.hq + head]);
    __syncthreads();
  }
  TileReads<E, DH> o;
  o.init();
  const uint32_t kb = lds0 + w * 2 * BYTES, vb = kb + BYTES;
  f32x16 acc[DH / 32] = {};
  float m = NEG_INF, sum = 0.0f;
  const int nb32 = len / 32 + (len % 32 != 0), step = 4 * a.splits;   // (lengths up to 2^31 - 1)
  // copies of 64 lanes
  constexpr int PT = 32 * TileRows<E, DH>::CPR / 64;
  u32x4 rk[PT], rv[PT];
  auto fetch = [&](int blk) {
#pragma unroll
    for (int x = 0; x < PT; ++x) {
      const int i = x * 64 + l, row = blk * 32 + i / TileRows<E, DH>::CPR, c = i % TileRows<E, DH>::CPR;
      rk[x] = rv[x] = u32x4{0u, 0u, 0u, 0u};
      if (row < len && c < cpr) {
        rk[x] = *reinterpret_cast<const u32x4*>(kh + row * a.ks + c * 16);
        rv[x] = *reinterpret_cast<const u32x4*>(vh + row * a.vs + c * 16);
      }
    }
  };
  int blk = split * 4 + w;
  if (blk < nb32) fetch(blk);
  for (; blk < nb32; blk += step) {
    wave_sync();
#pragma unroll
    for (int x = 0; x < PT; ++x) {
      const int i = x * 64 + l, row = i / TileRows<E, DH>::CPR, c = i % TileRows<E, DH>::CPR;
      const uint32_t at = row * RB + ((c ^ (row & TileRows<E, DH>::SWM)) << 4);
      lds_put(kb + at, rk[x]);
      lds_put(vb + at, rv[x]);
    }
    wave_sync();
    if (blk + step < nb32) fetch(blk + step);
    f32x16 x = block_of<E, DH>(o, kb, q);
    const int j0 = blk * 32, back = len - 1 - j0 - 4 * h;   // distance of the lane's key of row tile_row(v): back - tile_row(v)
    if (BIAS && len - 1 - j0 - 31 < a.dlast) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int bk = lds_at<uint8_t>(map + max(0, min(back - tile_row(v), a.dlast)));
        x[v] = fmaf(x[v], a.c, unit(a.bias[(int64_t)bk * a.hq + head]));
      }
    } else {
#pragma unroll
      for (int v = 0; v < 16; ++v) x[v] = BIAS ? fmaf(x[v], a.c, far) : x[v] * a.c;
    }
    if (len - j0 < 32) {
#pragma unroll
      for (int v = 0; v < 16; ++v) x[v] = back - tile_row(v) < 0 ? NEG_INF : x[v];
    }
    float bm = x[0];
#pragma unroll
    for (int v = 1; v < 16; ++v) bm = fmaxf(bm, x[v]);
    bm = fmaxf(bm, __shfl_xor(bm, 32));
    if (ballot(bm > m + (sizeof(E) == 2 ? 8.0f : 5.5f))) {
      const float up = fmaxf(m, bm);
      const float f = m == NEG_INF ? 0.0f : exp_of<E>(m - up);
      sum *= f;
#pragma unroll
      for (int nb = 0; nb < DH / 32; ++nb)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[nb][v] *= f;
      m = up;
    }
    const float ref = fmaxf(m, -NO_WEIGHT);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      x[v] = exp_of<E>(x[v] - ref);
      sum += x[v];
    }
    add_product<E, DH>(acc, x, o, vb);
  }
  sum += __shfl_xor(sum, 32);
  // the four waves: [4][group][P] of LDS, elements, then reference and sum
  __syncthreads();
  if (r < group) {
    const uint32_t at = lds0 + 4 * P * (w * group + r);
#pragma unroll
    for (int nb = 0; nb < DH / 32; ++nb)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        lds_put(at + 4 * (32 * nb + 8 * g + 4 * h),
                f32x4{acc[nb][4 * g], acc[nb][4 * g + 1], acc[nb][4 * g + 2], acc[nb][4 * g + 3]});
    if (h == 0) {
      lds_put<float>(at + 4 * DH, m);
      lds_put<float>(at + 4 * DH + 4, sum);
    }
  }
  __syncthreads();
  for (int t = tid; t < group * a.d; t += 256) {
    const int g = t / a.d, e = t % a.d;
    float top = -NO_WEIGHT, mm[4], all = 0.0f, val = 0.0f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      mm[x] = lds_at<float>(lds0 + 4 * (P * (x * group + g) + DH));
      top = fmaxf(top, mm[x]);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t at = lds0 + 4 * P * (x * group + g);
      const float f = exp_of<E>(mm[x] - top);
      all = fmaf(f, lds_at<float>(at + 4 * DH + 4), all);
      val = fmaf(f, lds_at<float>(at + 4 * e), val);
    }
    const int64_t row = (int64_t)u * a.hq + kvh * group + g;
    if (a.splits == 1) {
      const float y = all == 0.0f ? 0.0f : val / all;
      if constexpr (sizeof(E) == 2)
        reinterpret_cast<uint16_t*>(a.out)[row * a.d + e] = (uint16_t)pack_bf16(y, 0.0f);
      else
        reinterpret_cast<float*>(a.out)[row * a.d + e] = y;
    } else {
      a.part[(row * a.splits + split) * a.d + e] = val;
      if (e == 0) {
        float* p = a.part + ((int64_t)a.n_seq * a.hq * a.d + row * 2) * a.splits + split;
        p[0] = top;
        p[a.splits] = all;
      }
    }
  }
}

// A workgroup joins the parts of one head of one sequence: d columns x 1024 / d (or fewer) slices of the parts, whose
// factors are formed first.
template <class E>
__global__ __launch_bounds__(1024) void k_last_join(LastArgs a) {
  __shared__ float sv[1024], f[LAST_SPLITS], red[16];
  const int tid = threadIdx.x, slices = 1024 / a.d, e = tid % a.d, sl = tid / a.d;
  const float* p = a.part + (int64_t)blockIdx.x * a.splits * a.d;
  const float* stat = a.part + ((int64_t)a.n_seq * a.hq * a.d + (int64_t)blockIdx.x * 2) * a.splits;
  const float mine = tid < a.splits ? stat[tid] : -NO_WEIGHT, part = tid < a.splits ? stat[a.splits + tid] : 0.0f;
  float top = wave_max(mine);
  if (lane_id() == 0) red[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 16; ++q) top = fmaxf(top, red[q]);
  const float w = exp_of<E>(mine - top);
  if (tid < a.splits) f[tid] = w;
  const float some = wave_sumf(w * part);
  __syncthreads();
  if (lane_id() == 0) red[tid >> 6] = some;
  float val = 0.0f;
  if (sl < slices) {
#pragma unroll 8
    for (int s = sl; s < a.splits; s += slices) val = fmaf(f[s], p[(int64_t)s * a.d + e], val);
  }
  sv[tid] = val;
  __syncthreads();
  if (tid < a.d) {
    for (int s = 1; s < slices; ++s) val += sv[s * a.d + e];
    float all = 0.0f;
#pragma unroll
    for (int q = 0; q < 16; ++q) all += red[q];
    const float y = all == 0.0f ? 0.0f : val / all;
    const int64_t at = (int64_t)blockIdx.x * a.d + e;
    if constexpr (sizeof(E) == 2)
      reinterpret_cast<uint16_t*>(a.out)[at] = (uint16_t)pack_bf16(y, 0.0f);
    else
      reinterpret_cast<float*>(a.out)[at] = y;
  }
}

int slots_of(int64_t n, int64_t n_seq, int T) { return (int)(n / T + n_seq); }

// Waves of a workgroup of k_attn and k_attn_dq: four that share the tiles, or one by itself where a sequence has few more
// tokens than one wave's 32.  Measured (bf16, both kernels, one wave and four): 2,000 x 20 tokens, 4 heads of 64: 103 and
// 172 us; 200 x 200: 104 and 92; 16 x 1,021, 8 heads: 224 and 173; 1 x 4,000: 220 and 178.  The mean length decides, here and
// in key_waves (lengths lie on the device): among many short sequences a long one gets the short ones' form.
int query_waves(const rece_attention_config& c) { return c.n <= 64 * c.n_seq ? 1 : 4; }

// Waves of a workgroup of k_attn_dkv: more of them deal one tile's queries among themselves where there are too few tiles
// of keys to fill the card (two waves per SIMD, 2,048) and enough queries to deal.  Measured (bf16, with 1, 2, 4 waves):
// 4,000 tokens, 4 heads on 1: 674, 354, 183 us; 16 x 1,021, 8 heads on 2: 391, 272, 195; 200 x 200, 4 heads: 82, 96, 134.
// Eight where a CU has one tile at most, since one such workgroup fills it (4, 8 waves; tiles): 4,000 tokens (126): 183,
// 129 us; 4 x 600, 4 heads on 1 (79): 51, 38; 2 x 300, 4 heads (80): 14.9, 13.8; 8 x 400, 4 heads (432): 22, 27.
int key_waves(const rece_attention_config& c) {
  const int64_t tasks = (c.n / 32 + c.n_seq) * c.kv_heads, items = c.heads / c.kv_heads * (c.n / c.n_seq) / 64;
  const int most = tasks <= 256 ? 8 : tasks <= 1536 ? 4 : tasks <= 3000 ? 2 : 1;
  return items >= 4 ? most : items >= 2 ? std::min(most, 2) : 1;
}


// A launch with dynamic LDS (beyond 64 KB it has to be allowed first).
template <class A>
hipError_t launch(void (*kernel)(A), int64_t grid, int threads, size_t lds, hipStream_t st, const A& a) {
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<(unsigned)grid, threads, lds, st>>>(a);
  return hipGetLastError();
}

// f(type tag, padded head width, bias or not)
template <class F>
hipError_t attn_shape(bool bf16v, int d, bool bias, F f) {
  auto by_bias = [&](auto e, auto dh) { return bias ? f(e, dh, std::true_type()) : f(e, dh, std::false_type()); };
  auto by_width = [&](auto e) {
    if (d <= 32) return by_bias(e, std::integral_constant<int, 32>());
    if (d <= 64) return by_bias(e, std::integral_constant<int, 64>());
    return by_bias(e, std::integral_constant<int, 128>());
  };
  return bf16v ? by_width(bf16{}) : by_width(0.0f);
}

AttnArgs common_args(const rece_attention_config& c, const void* q, const void* k, const void* v, const int32_t* offs,
                     const float* bias) {
  AttnArgs a{};
  const int es = c.dtype == RECE_BF16 ? 2 : 4;
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.qs = c.q_stride * es;
  a.ks = c.k_stride * es;
  a.vs = c.v_stride * es;
  a.offs = offs;
  a.bias = bias;
  a.n = c.n;
  a.n_seq = (int)c.n_seq;
  a.d = c.d;
  a.hq = c.heads;
  a.hk = c.kv_heads;
  a.scale = c.scale;
  a.c = c.dtype == RECE_BF16 ? (float)((double)c.scale * 1.4426950408889634074) : c.scale;
  a.nbounds = bias ? c.n_bounds : 0;
  a.dlast = a.nbounds ? c.bounds[a.nbounds - 1] : 0;
  for (int t = 0; t <= RECE_MAX_BOUNDS; ++t) a.bounds[t] = t < a.nbounds ? c.bounds[t] : INT32_MAX;
  return a;
}

// Workspace: log-sum-exp [hq][n] float2, D [hq][n], bf16: what the outputs' rounding left, partial bias gradients.
struct AttnSpace {
  size_t lse, delta, low, part, total;
};
AttnSpace attn_space(const rece_attention_config& c) {
  AttnSpace s{};
  const size_t rows = (size_t)c.heads * c.n;
  s.lse = 0;
  s.delta = (rows * 8 + 15) & ~(size_t)15;
  s.low = (s.delta + rows * 4 + 15) & ~(size_t)15;
  s.part = s.low + (c.dtype == RECE_BF16 ? rows * c.d * 2 : 0);
  const size_t slots = (size_t)slots_of(c.n, c.n_seq, 32);
  s.total = s.part + slots * (c.n_bounds + 1) * c.heads * 4;
  return s;
}

}  // namespace

size_t attention_workspace_bytes(const rece_attention_config& c) { return attn_space(c).total; }

hipError_t attention_forward(const rece_attention_config& c, const void* q, const void* k, const void* v,
                             const int32_t* offs, const float* bias, void* ws, void* out, hipStream_t st) {
  AttnArgs a = common_args(c, q, k, v, offs, bias);
  a.out = static_cast<char*>(out);
  a.lse = static_cast<float2*>(ws);
  a.low = ws && c.dtype == RECE_BF16 ? static_cast<char*>(ws) + attn_space(c).low : nullptr;
  return attn_shape(c.dtype == RECE_BF16, c.d, bias != nullptr, [&](auto e, auto dh, auto bb) {
    const auto run = [&](auto nw) {
      using E = decltype(e);
      constexpr int DH = decltype(dh)::value, NW = decltype(nw)::value;
      constexpr bool B = decltype(bb)::value;
      using S = Shape<E, DH, NW>;
      a.slots = slots_of(c.n, c.n_seq, S::T);
      const size_t lds = 4 * S::BYTES + (B ? 4 * (a.dlast + 96) : 0);
      return launch(k_attn<E, DH, NW, B>, (int64_t)a.slots * a.hq + CLEAN, S::NT, lds, st, a);
    };
    return query_waves(c) == 1 ? run(std::integral_constant<int, 1>()) : run(std::integral_constant<int, 4>());
  });
}

hipError_t attention_backward(const rece_attention_config& c, const void* q, const void* k, const void* v,
                              const int32_t* offs, const float* bias, const void* out, void* ws, const void* dout,
                              void* dq, void* dk, void* dv, float* dbias, const int64_t (&strides)[3], hipStream_t st) {
  AttnArgs a = common_args(c, q, k, v, offs, bias);
  if (c.n == 0) return bias ? launch_join_rows(nullptr, 0, (a.nbounds + 1) * a.hq, dbias, st) : hipSuccess;
  const int es = c.dtype == RECE_BF16 ? 2 : 4;
  const AttnSpace sp = attn_space(c);
  a.out = const_cast<char*>(static_cast<const char*>(out));
  a.dout = static_cast<const char*>(dout);
  a.lse = static_cast<float2*>(ws);
  a.delta = reinterpret_cast<float*>(static_cast<char*>(ws) + sp.delta);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + sp.part);
  a.dq = static_cast<char*>(dq);
  a.dk = static_cast<char*>(dk);
  a.dv = static_cast<char*>(dv);
  a.dqs = strides[0] * es;
  a.dks = strides[1] * es;
  a.dvs = strides[2] * es;
  a.low = static_cast<char*>(ws) + sp.low;
  const int words = a.dlast + 96;
  hipError_t r = attn_shape(c.dtype == RECE_BF16, c.d, bias != nullptr, [&](auto e, auto dh, auto bb) {
    using E = decltype(e);
    constexpr int DH = decltype(dh)::value;
    constexpr bool B = decltype(bb)::value;
    const auto dq_run = [&](auto nw) {
      constexpr int NW = decltype(nw)::value;
      using S = Shape<E, DH, NW>;
      a.slots = slots_of(c.n, c.n_seq, S::T);
      const size_t lds = 4 * S::BYTES + (B ? 4 * words : 0);
      return launch(k_attn_dq<E, DH, NW, B>, (int64_t)a.slots * a.hq + CLEAN, S::NT, lds, st, a);
    };
    const hipError_t e1 =
        query_waves(c) == 1 ? dq_run(std::integral_constant<int, 1>()) : dq_run(std::integral_constant<int, 4>());
    if (e1 != hipSuccess) return e1;
    // as few waves as the tiles leave room for, as many heads' tables as then fit
    const int group = a.hq / a.hk;
    const auto lds_of = [&](int iw, int hp) {
      return (size_t)(iw * (2 * 32 * TileRows<E, DH>::RB + 3 * 128) + (B ? 4 * hp * (words + iw * (a.dlast + 34)) + iw * SKEW : 0));
    };
    // eight leave a lane 256 registers; four of float32 at 128 wide with a bias take 162 KB of LDS before its tables
    constexpr int MOST = sizeof(E) * DH <= 128 ? 8 : B && sizeof(E) * DH > 256 ? 2 : 4;
    int waves = std::min(key_waves(c), MOST);
    while (waves > 1 && lds_of(waves, 1) > MAX_LDS) waves /= 2;
    // (of up to four waves, more heads than this would cost the second workgroup of a CU)
    a.hp = 1;
    while (a.hp < group && lds_of(waves, a.hp + 1) <= std::max<size_t>(waves == 8 ? MAX_LDS : MAX_LDS / 2, lds_of(waves, 1))) ++a.hp;
    a.slots = slots_of(c.n, c.n_seq, 32);
    const auto dkv_run = [&](auto iw) {
      constexpr int IW = decltype(iw)::value;
      return launch(k_attn_dkv<E, DH, IW, B>, (int64_t)a.slots * a.hk + CLEAN, 64 * IW, lds_of(IW, a.hp), st, a);
    };
    return waves == 1 ? dkv_run(std::integral_constant<int, 1>())
                      : waves == 2 ? dkv_run(std::integral_constant<int, 2>())
                      : waves == 4 ? dkv_run(std::integral_constant<int, std::min(4, MOST)>())
                                   : dkv_run(std::integral_constant<int, MOST>());
  });
  if (r != hipSuccess || !bias) return r;
  return launch_join_rows(a.part, a.slots, (a.nbounds + 1) * a.hq, dbias, st);
}

// Parts of a sequence's keys: enough workgroups for two per CU, each wave with two blocks of 32 keys at least, and one
// part up to 1,024 keys (the join is another launch).  1 x 65,536, 2 key heads of 128: parts of 256 keys 23.4 us, of 512
// 24.3, of 1,024 33.2; 300 x 1,500: 512 workgroups 48 us, 1,024 53.
int64_t last_splits(const rece_attention_config& c, int64_t max_len) {
  if (max_len <= 1024) return 1;
  const int64_t wgs = c.n_seq * c.kv_heads, want = (512 + wgs - 1) / wgs, most = max_len / 256 + (max_len % 256 != 0);
  return std::max<int64_t>(1, std::min<int64_t>({want, most, LAST_SPLITS}));
}

size_t last_attention_workspace_bytes(const rece_attention_config& c, int64_t max_len) {
  const int64_t s = last_splits(c, max_len);
  return s == 1 ? 0 : (size_t)c.n_seq * c.heads * s * (c.d + 2) * 4;
}

hipError_t last_attention(const rece_attention_config& c, int64_t max_len, const void* q, const void* k, const void* v,
                          const int32_t* begin, const int32_t* length, const float* bias, void* ws, void* out,
                          hipStream_t st) {
  const int es = c.dtype == RECE_BF16 ? 2 : 4;
  LastArgs a{};
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.out = static_cast<char*>(out);
  a.qs = c.q_stride * es;
  a.ks = c.k_stride * es;
  a.vs = c.v_stride * es;
  a.begin = begin;
  a.length = length;
  a.bias = bias;
  a.part = static_cast<float*>(ws);
  a.rows = c.n;
  a.n_seq = (int)c.n_seq;
  a.d = c.d;
  a.hq = c.heads;
  a.hk = c.kv_heads;
  a.splits = (int)last_splits(c, max_len);
  a.c = c.dtype == RECE_BF16 ? (float)((double)c.scale * 1.4426950408889634074) : c.scale;
  a.nbounds = bias ? c.n_bounds : 0;
  a.dlast = a.nbounds ? c.bounds[a.nbounds - 1] : 0;
  for (int t = 0; t < a.nbounds; ++t) a.bounds[t] = c.bounds[t];
  return attn_shape(c.dtype == RECE_BF16, c.d, bias != nullptr, [&](auto e, auto dh, auto bb) {
    using E = decltype(e);
    constexpr int DH = decltype(dh)::value;
    constexpr bool B = decltype(bb)::value;
    const size_t lds = std::max<size_t>(8 * 32 * TileRows<E, DH>::RB, 16 * (a.hq / a.hk) * (DH + 4)) + (B ? a.dlast + 1 : 0);
    const hipError_t r = launch(k_last<E, DH, B>, c.n_seq * a.hk * a.splits, 256, lds, st, a);
    if (r != hipSuccess || a.splits == 1) return r;
    k_last_join<E><<<(unsigned)(c.n_seq * a.hq), 1024, 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace rece
