// Log-probability of one item per position under the softmax over the whole catalogue,
// its entropy, and their gradients (formulas in include/rece.h).  Every logit is formed
// on the matrix cores and consumed on chip; nothing of size s x C is stored.
//
// Logits are kept in base 2: x2_ij = X_i . Y_j * log2(e) / temperature, so that
// exp(x) = exp2(x2) takes one fma and one v_exp_f32 per logit.
//
// One kernel template sweeps "owners x streamed": a wave keeps OB blocks of 32 owner
// vectors in registers (the B operand of v_mfma_f32_32x32x16_bf16) and the other side
// passes through LDS in tiles, two buffers, the next tile's global loads issued before
// the current tile's work.  A block of 32 streamed x 32 owners leaves lane l with
// owner l % 32 and streamed rows 8 (v / 4) + 4 (l / 32) + v % 4, v = 0 .. 15, which is
// also the A-operand layout of the gradient product (k = streamed rows, in that order on
// both sides), so the weights never leave their registers; the streamed rows enter the
// second product transposed through the LDS transpose read.
//   LP_LSE (owners = positions, streamed = items): running sum of exp2(x2 - m)
//   LP_DX  (owners = positions, streamed = items): dX = G Y
//   LP_DY  (owners = items, streamed = positions): dY = G^T X
// The streamed side is cut into `splits` ranges, one workgroup each, when the owners
// alone would not fill the card; small kernels join the parts in a fixed order.
//
// Positions whose id is padding are left out first: the others are packed (rows, ids) in
// order into the workspace, so padding costs no products and nothing it holds (NaN or
// infinity) reaches a result.
#include <algorithm>
#include <cmath>

#include "rece_device.h"
#include "rece_internal.h"

namespace rece {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float LP_REF_LIMIT = 1.0995116e12f;   // 2^40: a block sum beyond it moves the reference
constexpr float LP_NEVER = 1e30f;               // lse2 of a row that has no weight: exp2(x2 - 1e30) = 0
constexpr int LP_ROW_PAD = 256;                 // packed rows are padded with zero rows to a multiple of this

enum LpMode { LP_LSE = 0, LP_DX = 1, LP_DY = 2 };

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Per packed row of the backward pass.
struct LpRow {
  float lse2, a, b, g;   // G = [hit] g - p (a + b (x2 - lse2)),  p = exp2(x2 - lse2)
};

struct LpArgs {
  const void* own;        // owner vectors [n_own][D]
  const void* str;        // streamed vectors [n_str][D]
  int64_t n_own, n_str;   // upper bounds; the positions' side is *nv
  const int32_t* nv;      // packed positions
  int own_is_pos;         // the owners are the packed positions (else the streamed side is)
  int splits;
  float c2;               // log2(e) / temperature
  float *m, *z, *t;       // LP_LSE: [splits][own_pad] reference, sum of 2^(x2 - m), sum of 2^(x2 - m) (x2 - m)
  int64_t own_pad;
  const LpRow* rows;      // gradients: of the packed positions
  const int32_t* idc;     // gradients: ids of the packed positions
  float* out;             // gradients: [splits][own_pad][D]
};

// Geometry of a streamed tile: TI rows of RB bytes; 16-byte chunk c of row n is stored at
// chunk c ^ (n & SWM), which spreads the 32 rows a fragment read touches over the banks.
template <class E, int D, int NWS> struct LpTile {
  static constexpr int RB = D * (int)sizeof(E);
  static constexpr int TI = NWS > 1 ? 32 * NWS : (RB <= 256 ? 64 : 32);
  static constexpr int CPR = RB / 16;
  static constexpr int SWM = (CPR < 8 ? CPR : 8) - 1;
  static constexpr int BYTES = TI * RB;
};

template <class E> struct LpMma;
template <> struct LpMma<bf16> {
  static __device__ __forceinline__ f32x16 run(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct LpMma<float> {   // four coordinates per chunk and lane half: four products of depth 2
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

// acc[nb] += G[32 owners][32 streamed] . rows[32 streamed][D], lane l holding G[owner l % 32]
// [streamed 8 (v / 4) + 4 (l / 32) + v % 4] in g[v].  bf16: G as the sum of NS bf16 terms (1: rounded
// once, for results that are themselves rounded to bf16; 3: all 24 bits).
template <class E, int D, int NWS, int NS>
__device__ __forceinline__ void lp_accumulate(f32x16 (&acc)[D / 32], const float (&g)[16], const char* tile, int rb) {
  using T = LpTile<E, D, NWS>;
  const int l = lane_id(), h = l >> 5;
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4 part[NS];
      float r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = g[8 * kk + e];
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const uint32_t w = pack_bf16(r[e], r[e + 1]);
          part[s][e / 2] = w;
          if (s + 1 < NS) {
            r[e] -= lo_f32(w);
            r[e + 1] -= hi_f32(w);
          }
        }
      // rows rb * 32 + 16 kk + 4 h + 0 .. 3 and + 8 .. 11, coordinates 32 nb + l % 32: within each
      // 16-lane group, source lane j names 4 coordinates of row j / 4
      const int j = l & 15, half = (l >> 4) & 1;
      const int row0 = rb * 32 + 16 * kk + 4 * h + (j >> 2), row1 = row0 + 8;
#pragma unroll
      for (int nb = 0; nb < D / 32; ++nb) {
        const int dim = 32 * nb + 16 * half + 4 * (j & 3);
        const char* a0 = tile + row0 * T::RB + (((dim >> 3) ^ (row0 & T::SWM)) << 4) + ((dim >> 2) & 1) * 8;
        const char* a1 = tile + row1 * T::RB + (((dim >> 3) ^ (row1 & T::SWM)) << 4) + ((dim >> 2) & 1) * 8;
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 b[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a0),
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a1)};
        const u32x4 bw = __builtin_bit_cast(u32x4, b);
#pragma unroll
        for (int s = 0; s < NS; ++s) acc[nb] = LpMma<bf16>::run(part[s], bw, acc[nb]);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int row = rb * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
#pragma unroll
      for (int nb = 0; nb < D / 32; ++nb) {
        const int dim = 32 * nb + (l & 31);
        const float b = *reinterpret_cast<const float*>(tile + row * T::RB + (((dim >> 2) ^ (row & T::SWM)) << 4) + 4 * (dim & 3));
        acc[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(g[v], b, acc[nb], 0, 0, 0);
      }
    }
  }
}

// NWO waves along the owners x NWS waves along a tile's rows; OB blocks of 32 owners per wave.
template <class E, int D, int OB, int NWO, int NWS, int MODE, bool ENT, int NS>
__global__ __launch_bounds__(64 * NWO * NWS) void k_lp_sweep(LpArgs a) {
  using T = LpTile<E, D, NWS>;
  constexpr int TI = T::TI, RB = T::RB, NT = 64 * NWO * NWS;
  constexpr int KC = RB / 32;              // 32-byte steps of a row: one chunk per lane half
  constexpr int PT = T::BYTES / 16 / NT;   // chunks a thread copies per tile
  static_assert(T::BYTES % (16 * NT) == 0, "whole chunks per thread");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, w = tid >> 6, l = lane_id(), h = l >> 5, r = l & 31;
  const int wo = w % NWO, ws = w / NWO;
  const int64_t nv = *a.nv;
  const int64_t n_own = a.own_is_pos ? nv : a.n_own, n_str = a.own_is_pos ? a.n_str : nv;
  const int64_t blk0 = (int64_t)blockIdx.x * (32 * OB * NWO), o0 = blk0 + wo * (32 * OB);
  const int split = blockIdx.y;
  if (blk0 >= n_own) return;
  const int64_t ntiles = (n_str + TI - 1) / TI, per = (ntiles + a.splits - 1) / a.splits;
  const int64_t tb = min(ntiles, (int64_t)split * per), te = min(ntiles, tb + per);

  u32x4 bown[OB][KC];
#pragma unroll
  for (int ob = 0; ob < OB; ++ob) {
    const int64_t o = min(o0 + 32 * ob + r, n_own - 1);
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.own) + o * RB);
#pragma unroll
    for (int t = 0; t < KC; ++t) bown[ob][t] = p[2 * t + h];
  }
  LpRow orow[OB];        // LP_DX
  int opos[OB];
  if constexpr (MODE == LP_DX) {
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      const int64_t o = min(o0 + 32 * ob + r, n_own - 1);
      orow[ob] = a.rows[o];
      opos[ob] = a.idc[o];
    }
  }
  float m[OB], z[OB], tt[OB];
  f32x16 acc[MODE == LP_LSE ? 1 : OB][D / 32];
#pragma unroll
  for (int ob = 0; ob < OB; ++ob) {
    m[ob] = NEG_INF;
    z[ob] = tt[ob] = 0.0f;
  }
  if constexpr (MODE != LP_LSE) {
#pragma unroll
    for (int ob = 0; ob < OB; ++ob)
#pragma unroll
      for (int nb = 0; nb < D / 32; ++nb)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[ob][nb][v] = 0.0f;
  }

  char* const bufs = smem;
  // streamed positions' constants and ids of a tile (LP_DY), behind the two tile buffers
  LpRow* const srow = reinterpret_cast<LpRow*>(smem + 2 * T::BYTES);
  int32_t* const sid = reinterpret_cast<int32_t*>(smem + 2 * T::BYTES + 2 * TI * sizeof(LpRow));
  u32x4 nxt[PT];
  u32x4 nrow = u32x4{0u, 0u, 0u, 0u};
  int nid = -1;
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      const int ch = q * NT + tid;
      const int64_t row = min(t * TI + ch / T::CPR, n_str - 1);
      nxt[q] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.str) + row * RB + (ch % T::CPR) * 16);
    }
    if constexpr (MODE == LP_DY) {
      if (tid < TI) {   // packed rows are padded with rows of no weight to whole tiles
        nrow = *reinterpret_cast<const u32x4*>(a.rows + t * TI + tid);
        nid = a.idc[t * TI + tid];
      }
    }
  };
  auto stash = [&](int64_t t) {
    char* buf = bufs + (t & 1) * T::BYTES;
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      const int ch = q * NT + tid, row = ch / T::CPR, c = ch % T::CPR;
      *reinterpret_cast<u32x4*>(buf + row * RB + ((c ^ (row & T::SWM)) << 4)) = nxt[q];
    }
    if constexpr (MODE == LP_DY) {
      if (tid < TI) {
        *reinterpret_cast<u32x4*>(srow + (t & 1) * TI + tid) = nrow;
        sid[(t & 1) * TI + tid] = nid;
      }
    }
  };
  if (tb < te) {
    fetch(tb);
    stash(tb);
  }
  for (int64_t t = tb; t < te; ++t) {
    __syncthreads();
    if (t + 1 < te) fetch(t + 1);
    const char* tile = bufs + (t & 1) * T::BYTES;
#pragma unroll 1
    for (int rb = ws; rb < TI / 32; rb += NWS) {
      const int64_t q0 = t * TI + rb * 32;
      const int lim = (int)min((int64_t)32, n_str - q0);   // rows of the block that exist (<= 0: none)
      f32x16 x[OB];
#pragma unroll
      for (int ob = 0; ob < OB; ++ob)
#pragma unroll
        for (int v = 0; v < 16; ++v) x[ob][v] = 0.0f;
      const int row = rb * 32 + r;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const u32x4 f = *reinterpret_cast<const u32x4*>(tile + row * RB + (((2 * k + h) ^ (row & T::SWM)) << 4));
#pragma unroll
        for (int ob = 0; ob < OB; ++ob) x[ob] = LpMma<E>::run(f, bown[ob][k], x[ob]);
      }
      if constexpr (MODE == LP_LSE) {
#pragma unroll
        for (int ob = 0; ob < OB; ++ob) {
          float e[16], d[16];
          auto sums = [&](float& s, float& st) {
            s = st = 0.0f;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const int n = 8 * (v >> 2) + 4 * h + (v & 3);
              d[v] = fmaf(x[ob][v], a.c2, -m[ob]);
              e[v] = exp2_fast(d[v]);
              if (lim < 32 && n >= lim) e[v] = d[v] = 0.0f;
              s += e[v];
              if constexpr (ENT) st = fmaf(e[v], d[v], st);
            }
          };
          float s, st;
          sums(s, st);
          // the reference m is the first block's maximum and moves only when a block's sum
          // would pass 2^40 (exp2 has the range); NaN logits end here too, and stay NaN
          if (ballot(!(s < LP_REF_LIMIT))) {
            float bm = NEG_INF;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const int n = 8 * (v >> 2) + 4 * h + (v & 3);
              if (lim >= 32 || n < lim) bm = fmaxf(bm, x[ob][v] * a.c2);
            }
            if (bm > m[ob]) {
              const float f = z[ob] > 0.0f ? exp2_fast(m[ob] - bm) : 0.0f;
              if constexpr (ENT) tt[ob] = z[ob] > 0.0f ? (tt[ob] + z[ob] * (m[ob] - bm)) * f : 0.0f;
              z[ob] *= f;
              m[ob] = bm;
            }
            sums(s, st);
          }
          if (m[ob] != NEG_INF) {
            z[ob] += s;
            if constexpr (ENT) tt[ob] += st;
          }
        }
      } else {
        bool hit = false;
        if constexpr (MODE == LP_DX) {
#pragma unroll
          for (int ob = 0; ob < OB; ++ob) hit = hit || (opos[ob] >= q0 && opos[ob] < q0 + 32);
        } else {
          const int id = sid[(t & 1) * TI + row];
          hit = id >= o0 && id < o0 + 32 * OB;
        }
        const bool any = ballot(hit) != 0;
#pragma unroll
        for (int ob = 0; ob < OB; ++ob) {
          float g[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int n = 8 * (v >> 2) + 4 * h + (v & 3);
            LpRow c;
            if constexpr (MODE == LP_DX)
              c = orow[ob];
            else
              c = srow[(t & 1) * TI + rb * 32 + n];
            const float d = fmaf(x[ob][v], a.c2, -c.lse2);
            const float wgt = ENT ? fmaf(c.b, d, c.a) : c.a;
            g[v] = -exp2_fast(d) * wgt;
            if (lim < 32 && n >= lim) g[v] = 0.0f;
            if (any) {
              bool on;
              if constexpr (MODE == LP_DX)
                on = q0 + n == opos[ob];
              else
                on = (int64_t)sid[(t & 1) * TI + rb * 32 + n] == o0 + 32 * ob + r;
              if (on) g[v] += c.g;
            }
          }
          // a block that holds some row's own item: 1 - p would lose its digits in one bf16 term
          if (any)
            lp_accumulate<E, D, NWS, 3>(acc[ob], g, tile, rb);
          else
            lp_accumulate<E, D, NWS, NS>(acc[ob], g, tile, rb);
        }
      }
    }
    if (t + 1 < te) stash(t + 1);
  }

  if constexpr (MODE == LP_LSE) {
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      // the two lane halves hold different rows of the same owner
      const float om = __shfl_xor(m[ob], 32), oz = __shfl_xor(z[ob], 32), ot = __shfl_xor(tt[ob], 32);
      const float mm = fmaxf(m[ob], om);
      const float f0 = m[ob] == NEG_INF ? 0.0f : exp2_fast(m[ob] - mm), f1 = om == NEG_INF ? 0.0f : exp2_fast(om - mm);
      const float zz = z[ob] * f0 + oz * f1;
      const float t0 = m[ob] == NEG_INF ? 0.0f : (tt[ob] + z[ob] * (m[ob] - mm)) * f0;
      const float t1 = om == NEG_INF ? 0.0f : (ot + oz * (om - mm)) * f1;
      const int64_t o = o0 + 32 * ob + r;
      if (h == 0 && o < n_own) {
        const int64_t at = ((int64_t)split * NWS + ws) * a.own_pad + o;
        a.m[at] = mm;
        a.z[at] = zz;
        if constexpr (ENT) a.t[at] = t0 + t1;
      }
    }
  } else {
    float* out = a.out + ((int64_t)split * NWS + ws) * a.own_pad * D;
#pragma unroll
    for (int ob = 0; ob < OB; ++ob)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t o = o0 + 32 * ob + 8 * (v >> 2) + 4 * h + (v & 3);
        if (o < n_own)
#pragma unroll
          for (int nb = 0; nb < D / 32; ++nb) out[o * D + 32 * nb + r] = acc[ob][nb][v];
      }
  }
}

// ------------------------------------------------------------------ packing
// One workgroup: the positions with an id in [0, C), in order.  inv[i] is position i's
// place among them, or -1.
constexpr int PACK_THREADS = 1024;
__global__ __launch_bounds__(PACK_THREADS) void k_lp_list(const int32_t* __restrict__ ids, int64_t s, int64_t C,
                                                          int32_t* __restrict__ nv, int32_t* __restrict__ list,
                                                          int32_t* __restrict__ inv) {
  constexpr int PER = 8;   // ids per thread and step, loaded before the step's prefix sum
  __shared__ int32_t wsum[PACK_THREADS / WAVE];
  const int tid = threadIdx.x, w = tid >> 6, l = lane_id();
  int64_t done = 0;
  for (int64_t b = 0; b < s; b += PACK_THREADS * PER) {
    const int64_t i0 = b + (int64_t)tid * PER;
    uint32_t ok = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int id = i0 + q < s ? ids[i0 + q] : -1;
      ok |= id >= 0 && id < C ? 1u << q : 0u;
    }
    const int mine = __popc(ok);
    const int incl = (int)wave_prefix_incl((uint32_t)mine);
    __syncthreads();
    if (l == WAVE - 1) wsum[w] = incl;
    __syncthreads();
    int64_t at = done + incl - mine;
    int tot = 0;
#pragma unroll
    for (int q = 0; q < PACK_THREADS / WAVE; ++q) {
      if (q < w) at += wsum[q];
      tot += wsum[q];
    }
    done += tot;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (i0 + q >= s) break;
      const bool on = (ok >> q) & 1u;
      inv[i0 + q] = on ? (int32_t)at : -1;
      if (on) list[at++] = (int32_t)(i0 + q);
    }
  }
  if (tid == 0) *nv = (int32_t)done;
}

// Packed rows and ids (zero rows up to the padding), and the base-2 logit of each row's
// own item.  One lane group of D / (16 / sizeof(E)) lanes per row.
template <class E, int D>
__global__ __launch_bounds__(256) void k_lp_pack(const E* __restrict__ X, const E* __restrict__ Y,
                                                 const int32_t* __restrict__ ids, const int32_t* __restrict__ nv_p,
                                                 const int32_t* __restrict__ list, int64_t pad, float c2,
                                                 E* __restrict__ Xc, int32_t* __restrict__ idc, float* __restrict__ own2) {
  constexpr int EPL = 16 / (int)sizeof(E), LPR = D / EPL;
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int sub = threadIdx.x % LPR;
  const int64_t nv = *nv_p;
  if (row >= min(pad, (nv + LP_ROW_PAD - 1) / LP_ROW_PAD * LP_ROW_PAD)) return;
  u32x4 x = u32x4{0u, 0u, 0u, 0u};
  int id = -1;
  float dot = 0.0f;
  if (row < nv) {
    const int64_t i = list[row];
    id = ids[i];
    x = reinterpret_cast<const u32x4*>(X + i * D)[sub];
    const u32x4 y = reinterpret_cast<const u32x4*>(Y + (int64_t)id * D)[sub];
    const E* xe = reinterpret_cast<const E*>(&x);
    const E* ye = reinterpret_cast<const E*>(&y);
#pragma unroll
    for (int t = 0; t < EPL; ++t) dot = fmaf(to_f32(xe[t]), to_f32(ye[t]), dot);
  }
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
  reinterpret_cast<u32x4*>(Xc + row * D)[sub] = x;
  if (sub == 0) {
    idc[row] = id;
    own2[row] = dot * c2;
  }
}

// ------------------------------------------------------------------ joins
// Per position: the parts of its sum, in order -> log-sum-exp, log-probability, entropy.
__global__ __launch_bounds__(256) void k_lp_finish(const int32_t* __restrict__ inv, int64_t s, int parts, int64_t pad,
                                                   const float* __restrict__ m, const float* __restrict__ z,
                                                   const float* __restrict__ t, const float* __restrict__ own2,
                                                   float* __restrict__ lse2, float* __restrict__ ent_c,
                                                   float* __restrict__ logp, float* __restrict__ entropy) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= s) return;
  const int64_t r = inv[i];
  if (r < 0) {
    logp[i] = 0.0f;
    if (entropy) entropy[i] = 0.0f;
    return;
  }
  float mm = NEG_INF;
  for (int p = 0; p < parts; ++p) mm = fmaxf(mm, m[(int64_t)p * pad + r]);
  float zz = 0.0f, tt = 0.0f;
  for (int p = 0; p < parts; ++p) {
    const float mp = m[(int64_t)p * pad + r], zp = z[(int64_t)p * pad + r];
    if (mp == NEG_INF) continue;
    const float f = exp2_fast(mp - mm);
    zz = fmaf(zp, f, zz);
    if (entropy) tt += (t[(int64_t)p * pad + r] + zp * (mp - mm)) * f;
  }
  const float lz = log2f(zz), l2 = mm + lz;
  lse2[r] = l2;
  logp[i] = (own2[r] - l2) * LN2;
  if (entropy) {
    const float H = (lz - tt / zz) * LN2;
    entropy[i] = H;
    ent_c[r] = H;
  }
}

// Constants of the gradient per packed row; rows of no weight up to the padding.
__global__ __launch_bounds__(256) void k_lp_coef(const int32_t* __restrict__ nv_p, const int32_t* __restrict__ list,
                                                 int64_t pad, const float* __restrict__ lse2,
                                                 const float* __restrict__ ent_c, const float* __restrict__ dlogp,
                                                 const float* __restrict__ dent, float inv_t, LpRow* __restrict__ rows) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= pad) return;
  LpRow c{LP_NEVER, 0.0f, 0.0f, 0.0f};
  if (r < *nv_p) {
    const int64_t i = list[r];
    const float g = dlogp[i] * inv_t, h = dent ? dent[i] * inv_t : 0.0f;
    c.lse2 = lse2[r];
    c.g = g;
    c.a = dent ? fmaf(h, ent_c[r], g) : g;
    c.b = h * LN2;
  }
  rows[r] = c;
}

// out row = sum of the parts' rows, in order; inv: row of the parts for each output row (or -1: zeros).
template <bool B16>
__global__ __launch_bounds__(256) void k_lp_join(const float* __restrict__ part, int parts, int64_t pad, int d,
                                                 const int32_t* __restrict__ inv, int64_t n, void* __restrict__ out) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = d / 4;
  if (q >= n * per) return;
  const int64_t i = q / per;
  const int c = (int)(q % per) * 4;
  const int64_t r = inv ? inv[i] : i;
  float4 v = float4{0.0f, 0.0f, 0.0f, 0.0f};
  if (r >= 0) {
    for (int p = 0; p < parts; ++p) {
      const float4 w = *reinterpret_cast<const float4*>(part + ((int64_t)p * pad + r) * d + c);
      v = float4{v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w};
    }
  }
  if constexpr (B16) {
    uint2 o;
    o.x = pack_bf16(v.x, v.y);
    o.y = pack_bf16(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i * d + c) = o;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + i * d + c) = v;
  }
}

// ------------------------------------------------------------------ host side
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Splits of the streamed side: enough workgroups to fill the card (256 CUs, a few each),
// no split shorter than a few tiles, and the parts within 256 MB.
constexpr int64_t LP_TARGET_BLOCKS = 1024;
constexpr int64_t LP_MIN_TILES = 4;
constexpr int64_t LP_PART_BYTES = (int64_t)256 << 20;
int lp_splits(int64_t n_own, int64_t own_block, int64_t n_str, int64_t ti, int64_t part_bytes) {
  const int64_t nb = ceil_div(n_own, own_block);
  int64_t sp = LP_TARGET_BLOCKS / nb;
  sp = std::min(sp, ceil_div(n_str, ti) / LP_MIN_TILES);
  sp = std::min(sp, LP_PART_BYTES / std::max<int64_t>(part_bytes, 1));
  return (int)std::max<int64_t>(1, std::min<int64_t>(sp, 4096));
}

template <class E, int D> struct LpShape {
  static constexpr int OB_LSE = sizeof(E) == 2 && D <= 128 ? 2 : 1;
  static constexpr int OB_GRAD = 1;
  static constexpr int NWO = 4;
};

struct LpLayout {
  int64_t pad;
  size_t nv, list, inv, idc, own2, lse2, ent, rows, xc, m, z, t, dx, dy, bytes;
  int sp_lse, sp_dx, sp_dy;
};

template <class E, int D>
LpLayout lp_layout_t(int64_t s, int64_t C, uint32_t flags) {
  using S = LpShape<E, D>;
  using T = LpTile<E, D, 1>;
  LpLayout y{};
  y.pad = ceil_div(s, LP_ROW_PAD) * LP_ROW_PAD;
  y.sp_lse = lp_splits(s, 32 * S::OB_LSE * S::NWO, C, T::TI, 12 * y.pad);
  y.sp_dx = lp_splits(s, 32 * S::OB_GRAD * S::NWO, C, T::TI, y.pad * D * 4);
  y.sp_dy = lp_splits(C, 32 * S::OB_GRAD * S::NWO, s, T::TI, C * D * 4);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  y.nv = take(16);
  y.list = take(y.pad * 4);
  y.inv = take(y.pad * 4);
  y.idc = take(y.pad * 4);
  y.own2 = take(y.pad * 4);
  y.lse2 = take(y.pad * 4);
  y.ent = take(flags & RECE_FLAG_ENTROPY ? y.pad * 4 : 0);
  y.xc = take((size_t)y.pad * D * sizeof(E));
  // what one call alone uses: the forward pass's parts, the backward pass's rows and parts
  const size_t base = off;
  const size_t parts = (size_t)y.sp_lse * y.pad * 4;
  y.m = take(parts);
  y.z = take(parts);
  y.t = take(flags & RECE_FLAG_ENTROPY ? parts : 0);
  const size_t fwd = off;
  off = base;
  if (!(flags & RECE_FLAG_NO_GRAD)) {
    y.rows = take(y.pad * sizeof(LpRow));
    // dX is finished before the dY sweep starts
    y.dx = y.dy = take(std::max((size_t)y.sp_dx * y.pad * D * 4, (size_t)y.sp_dy * C * D * 4));
  }
  y.bytes = std::max(fwd, off);
  return y;
}

template <class E, int D, int OB, int NWO, int NWS, int MODE, bool ENT, int NS>
hipError_t lp_launch(const LpArgs& a, int64_t n_own, hipStream_t st) {
  using T = LpTile<E, D, NWS>;
  const size_t lds = 2 * (size_t)T::BYTES + (MODE == LP_DY ? 2 * T::TI * (sizeof(LpRow) + 4) : 0);
  auto kern = k_lp_sweep<E, D, OB, NWO, NWS, MODE, ENT, NS>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)ceil_div(n_own, 32 * OB * NWO), (unsigned)a.splits);
  hipLaunchKernelGGL(kern, grid, dim3(64 * NWO * NWS), lds, st, a);
  return hipGetLastError();
}

#define LP_TRY(call)                     \
  do {                                   \
    const hipError_t e_ = (call);        \
    if (e_ != hipSuccess) return e_;     \
  } while (0)

template <class T> T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

template <class E, int D>
hipError_t lp_forward_t(int64_t s, int64_t C, float temperature, uint32_t flags, const void* X, const void* Y,
                        const int32_t* ids, void* ws, float* logp, float* entropy, hipStream_t st) {
  using S = LpShape<E, D>;
  const LpLayout y = lp_layout_t<E, D>(s, C, flags);
  const float c2 = LOG2E / temperature;
  hipLaunchKernelGGL(k_lp_list, dim3(1), dim3(PACK_THREADS), 0, st, ids, s, C, at<int32_t>(ws, y.nv),
                     at<int32_t>(ws, y.list), at<int32_t>(ws, y.inv));
  LP_TRY(hipGetLastError());
  const int64_t lanes = y.pad * (D * (int)sizeof(E) / 16);
  hipLaunchKernelGGL((k_lp_pack<E, D>), dim3((unsigned)ceil_div(lanes, 256)), dim3(256), 0, st,
                     static_cast<const E*>(X), static_cast<const E*>(Y), ids, at<int32_t>(ws, y.nv),
                     at<int32_t>(ws, y.list), y.pad, c2, at<E>(ws, y.xc), at<int32_t>(ws, y.idc), at<float>(ws, y.own2));
  LP_TRY(hipGetLastError());
  LpArgs a{};
  a.own = at<E>(ws, y.xc);
  a.str = Y;
  a.n_own = s;
  a.n_str = C;
  a.nv = at<int32_t>(ws, y.nv);
  a.own_is_pos = 1;
  a.splits = y.sp_lse;
  a.c2 = c2;
  a.m = at<float>(ws, y.m);
  a.z = at<float>(ws, y.z);
  a.t = at<float>(ws, y.t);
  a.own_pad = y.pad;
  if (entropy)
    LP_TRY((lp_launch<E, D, S::OB_LSE, S::NWO, 1, LP_LSE, true, 1>(a, s, st)));
  else
    LP_TRY((lp_launch<E, D, S::OB_LSE, S::NWO, 1, LP_LSE, false, 1>(a, s, st)));
  hipLaunchKernelGGL(k_lp_finish, dim3((unsigned)ceil_div(s, 256)), dim3(256), 0, st, at<int32_t>(ws, y.inv), s, y.sp_lse,
                     y.pad, a.m, a.z, a.t, at<float>(ws, y.own2), at<float>(ws, y.lse2), at<float>(ws, y.ent), logp,
                     entropy);
  return hipGetLastError();
}

template <class E, int D, bool ENT, int NS>
hipError_t lp_backward_g(int64_t s, int64_t C, float temperature, uint32_t flags, const void* Y, void* ws,
                         const float* dlogp, const float* dent, void* dX, void* dY, hipStream_t st) {
  using S = LpShape<E, D>;
  const LpLayout y = lp_layout_t<E, D>(s, C, flags);
  hipLaunchKernelGGL(k_lp_coef, dim3((unsigned)ceil_div(y.pad, 256)), dim3(256), 0, st, at<int32_t>(ws, y.nv),
                     at<int32_t>(ws, y.list), y.pad, at<float>(ws, y.lse2), at<float>(ws, y.ent), dlogp, dent,
                     1.0f / temperature, at<LpRow>(ws, y.rows));
  LP_TRY(hipGetLastError());
  LpArgs a{};
  a.nv = at<int32_t>(ws, y.nv);
  a.c2 = LOG2E / temperature;
  a.rows = at<LpRow>(ws, y.rows);
  a.idc = at<int32_t>(ws, y.idc);
  auto join = [&](const int32_t* inv, int64_t n, void* out) {
    const dim3 grid((unsigned)ceil_div(n * (D / 4), 256));
    if (flags & RECE_FLAG_BF16_GRADS)
      hipLaunchKernelGGL((k_lp_join<true>), grid, dim3(256), 0, st, a.out, a.splits, a.own_pad, D, inv, n, out);
    else
      hipLaunchKernelGGL((k_lp_join<false>), grid, dim3(256), 0, st, a.out, a.splits, a.own_pad, D, inv, n, out);
    return hipGetLastError();
  };
  a.own = at<E>(ws, y.xc);
  a.str = Y;
  a.n_own = s;
  a.n_str = C;
  a.own_is_pos = 1;
  a.splits = y.sp_dx;
  a.own_pad = y.pad;
  a.out = at<float>(ws, y.dx);
  LP_TRY((lp_launch<E, D, S::OB_GRAD, S::NWO, 1, LP_DX, ENT, NS>(a, s, st)));
  LP_TRY(join(at<int32_t>(ws, y.inv), s, dX));
  a.own = Y;
  a.str = at<E>(ws, y.xc);
  a.n_own = C;
  a.n_str = s;
  a.own_is_pos = 0;
  a.splits = y.sp_dy;
  a.own_pad = C;
  a.out = at<float>(ws, y.dy);
  LP_TRY((lp_launch<E, D, S::OB_GRAD, S::NWO, 1, LP_DY, ENT, NS>(a, C, st)));
  return join(nullptr, C, dY);
}

template <class E, int D>
hipError_t lp_backward_t(int64_t s, int64_t C, float temperature, uint32_t flags, const void* Y, void* ws,
                         const float* dlogp, const float* dent, void* dX, void* dY, hipStream_t st) {
  // bf16 results take one bf16 term of G, float32 results all of its bits
  const bool one = flags & RECE_FLAG_BF16_GRADS;
  if (dent) {
    if (one) return lp_backward_g<E, D, true, 1>(s, C, temperature, flags, Y, ws, dlogp, dent, dX, dY, st);
    return lp_backward_g<E, D, true, 3>(s, C, temperature, flags, Y, ws, dlogp, dent, dX, dY, st);
  }
  if (one) return lp_backward_g<E, D, false, 1>(s, C, temperature, flags, Y, ws, dlogp, dent, dX, dY, st);
  return lp_backward_g<E, D, false, 3>(s, C, temperature, flags, Y, ws, dlogp, dent, dX, dY, st);
}

}  // namespace

#define LP_SIZES(E, CALL)        \
  switch (d) {                   \
    case 32: return CALL(E, 32); \
    case 64: return CALL(E, 64); \
    case 128: return CALL(E, 128); \
    default: return CALL(E, 256); \
  }

size_t logprob_workspace_bytes(bool bf16v, int64_t s, int64_t C, int d, uint32_t flags) {
#define LP_CALL(E, D) lp_layout_t<E, D>(s, C, flags).bytes
  if (bf16v) LP_SIZES(bf16, LP_CALL)
  LP_SIZES(float, LP_CALL)
#undef LP_CALL
}

hipError_t logprob_forward(bool bf16v, int64_t s, int64_t C, int d, float temperature, uint32_t flags, const void* X,
                           const void* Y, const int32_t* ids, void* ws, float* logp, float* entropy, hipStream_t st) {
#define LP_CALL(E, D) lp_forward_t<E, D>(s, C, temperature, flags, X, Y, ids, ws, logp, entropy, st)
  if (bf16v) LP_SIZES(bf16, LP_CALL)
  LP_SIZES(float, LP_CALL)
#undef LP_CALL
}

hipError_t logprob_backward(bool bf16v, int64_t s, int64_t C, int d, float temperature, uint32_t flags, const void* X,
                            const void* Y, const int32_t* ids, void* ws, const float* dlogp, const float* dentropy,
                            void* dX, void* dY, hipStream_t st) {
  (void)X;
  (void)ids;   // the workspace holds the packed rows and ids
#define LP_CALL(E, D) lp_backward_t<E, D>(s, C, temperature, flags, Y, ws, dlogp, dentropy, dX, dY, st)
  if (bf16v) LP_SIZES(bf16, LP_CALL)
  LP_SIZES(float, LP_CALL)
#undef LP_CALL
}

}  // namespace rece
