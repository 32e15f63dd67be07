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
//   LP_LSE  (owners = positions, streamed = items): sum of exp2(x2 - m), and with it the entropy's
//   LP_LSEO (the same, before gradients without entropies): and the sums of item rows, so that dX
//           needs no sweep of its own
//   LP_DX   (owners = positions, streamed = items): dX = G Y, with entropies
//   LP_DY   (owners = items, streamed = positions): dY = G^T X
// The work is dealt to a grid that fills the card once (rece_parts.h); small kernels join the parts
// in a fixed order.
//
// What bounds it: the exponential of each logit (v_exp_f32, about 9 cycles of a SIMD for 64 logits, with 2
// to 4 cheaper instructions beside it), the split of each weight into bf16 terms (6 more), and the products share a
// SIMD's issue: at d 64 vector and matrix units are busy 67 % and 46 % of LP_LSEO, 57 % and 39 % of LP_DY (popular
// items meet their own positions in most tiles); at d 256 waves wait more than half of their cycles (two per SIMD,
// registers spilled).  Measured (bf16 vectors; products counted with both terms of a weight):
//   51,200 (a quarter padding) x 30,000 x 64  with bf16 gradients 935 us: LP_LSEO 507 and LP_DY 571 us alone (870 and
//                          775 TFLOP/s, 2.0e12 exponentials a second and more), packing and joins 45 us; with float32
//                          gradients (three terms) 1,293 us
//   4,099 (a tenth padding) x 50,021 x 256  with entropies and bf16 gradients 771 us: LP_LSE 124, LP_DX 292,
//                          LP_DY 407 us alone (760, 970, 700 TFLOP/s); with float32 gradients 985 us
//   8,192 (a tenth padding) x 30,000 x 128  with bf16 gradients 374 us: LP_LSEO 187, LP_DY 209 us alone
//   40 (a tenth padding) x 1,000,000 x 64  with bf16 gradients 301 us: LP_LSEO 43, LP_DY 86, the join of its float32
//                          parts 111, of the 3,000 parts of 36 positions 60 us
//   2,047 (a tenth padding) x 200,000 x 128  log-probabilities 121 us: LP_LSE 118 us (800 TFLOP/s)
//   5 x 1,000,000 x 64     log-probabilities and entropies 40 us: LP_LSE 26 us, 128 MB at 4.9 TB/s
//   256 x 2,000 x 64 float32 with entropies and gradients 50 us: eight launches of 2 to 12 us
//   636 (a tenth padding) x 30,018 x 256 float32 with gradients 564 us: LP_LSEO 275, LP_DY 272 us (64 TFLOP/s of
//                          154: one wave per SIMD); 2,047 x 30,018 x 64 log-probabilities 89 us (85: 83 TFLOP/s)
//
// Positions whose id is padding are left out first: the others are packed (rows, ids) in
// order into the workspace, so padding costs no products and nothing it holds (NaN or
// infinity) reaches a result.
#include <algorithm>
#include <cmath>

#include "rece_device.h"
#include "rece_ops.h"
#include "rece_parts.h"
#include "rece_tile.h"

namespace rece {

namespace {

constexpr float LN2 = 0.6931471805599453f;
constexpr float LP_REF_LIMIT = 1.1529215e18f;   // 2^60: a sum beyond it is taken again with a better reference
constexpr float LP_FLOOR = -1e28f;              // a reference where no logit is: those beyond the end lie at -1e30
constexpr float LP_NEVER = 1e30f;               // lse2 of a row that has no weight: exp2(x2 - 1e30) = 0
constexpr int LP_FRAGS = 4;                     // fragments of a row read ahead of their products
constexpr int LP_ROW_PAD = 256;                 // packed rows are padded with zero rows to a multiple of this

enum LpMode { LP_LSE = 0, LP_LSEO = 1, LP_DX = 2, LP_DY = 3 };

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Per packed row of the backward pass.
struct LpRow {
  float lse2, a, b, g;   // G = g for the row's own item, -p (a + b (x2 - lse2)) for others, p = exp2(x2 - lse2)
};

// log2(e) / temperature: rounded, and what the rounding left.  Its error would scale every logit alike, 6e-8 of a
// logit's distance from the others, which is the relative error of 1 - p where p is near 1.  The second term is
// taken for float32 inputs (their sweeps wait for the products, not for it); with bf16 inputs it is 0.
struct LpScale {
  float hi, lo;
};

struct LpArgs {
  const void* own;        // owner vectors [n_own][D]
  const void* str;        // streamed vectors [n_str][D]
  SweepParts parts;       // sizes, workgroups, and where parts lie
  LpScale c2;             // log2(e) / temperature
  float4* stat;           // LP_LSE(O): parts (reference m, sum of 2^(x2 - m), sum of 2^(x2 - m) (x2 - m), 0)
  const LpRow* rows;      // LP_DX, LP_DY: of the packed positions (LP_DY: padded with rows of no weight)
  const int32_t* idc;     // ids of the packed positions
  float* out;             // LP_LSEO, LP_DX, LP_DY: parts.rows
  int terms;              // bf16 terms of a weight in the products (2 or 3; 1 with float32 inputs)
};

// Geometry of a streamed tile: TI rows of RB bytes; 16-byte chunk c of row n is stored at
// chunk c ^ (n & SWM), which spreads the 32 rows a fragment read touches over the banks.
template <class E, int D, int NWS> struct LpTile {
  static constexpr int RB = D * (int)sizeof(E);
  static constexpr int TI = NWS > 1 ? 32 * NWS : (RB <= 128 ? 128 : RB <= 256 ? 64 : 32);
  static constexpr int CPR = RB / 16;
  static constexpr int SWM = (CPR < 8 ? CPR : 8) - 1;
  static constexpr int BYTES = TI * RB;
};

template <class E> using LpMma = TileMma<E>;

// Two floats as two bf16 terms each.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  const float ra = a - lo_f32(hi), rb = b - hi_f32(hi);
  lo = pack_bf16(ra, rb);
}

// x log2(e) / temperature - r (the small term last, onto the difference)
template <bool LO>
__device__ __forceinline__ float lp_less(float x, LpScale c, float r) {
  const float d = fmaf(x, c.hi, -r);
  return LO ? fmaf(x, c.lo, d) : d;
}

// Gradient by a logit of another item: -p (a + b d) with d = x2 - lse2, p = 2^d.
template <bool ENT>
__device__ __forceinline__ float lp_weight(float d, float a, float b) {
  return -exp2_fast(d) * (ENT ? fmaf(b, d, a) : a);
}

// Row of value v of a 32 x 32 block (less 4 h for the lane half h).
__device__ __forceinline__ constexpr int lp_row(int v) { return tile_row(v); }

// acc[ob][nb] += G[32 owners][32 streamed] . rows[32 streamed][D], lane l holding G[owner l % 32]
// [streamed lp_row(v) + 4 (l / 32)] in g[ob][v].  bf16: TERMS products, each with the bf16
// rounding of what the ones before left of G (2: off by at most 2^-16 of a weight, 3: all 24 bits).
template <class E, int D, int NWS, int OB, int TERMS>
__device__ __forceinline__ void lp_product(f32x16 (&acc)[OB][D / 32], f32x16 (&g)[OB], const TileReads<E, D>& o,
                                           uint32_t base) {
  using T = LpTile<E, D, NWS>;
  if constexpr (sizeof(E) == 2) {
    auto term = [&](u32x4 (&part)[OB][2]) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[ob][kk][e] = pack_bf16(g[ob][8 * kk + 2 * e], g[ob][8 * kk + 2 * e + 1]);
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb) {
          const uint32_t at = o.y[nb % o.NY] + base + (nb / o.NY) * 128 + 16 * kk * T::RB;
          const s16x4 b[2] = {lds_tr4(at), lds_tr4(at + 8 * T::RB)};
          const u32x4 bw = __builtin_bit_cast(u32x4, b);
#pragma unroll
          for (int ob = 0; ob < OB; ++ob) acc[ob][nb] = LpMma<bf16>::run(part[ob][kk], bw, acc[ob][nb]);
        }
      }
    };
    if constexpr (TERMS == 2) {   // both terms against the same fragments: each row of the tile is read once
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        u32x4 hi[OB], lo[OB];
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t first, second;
            split_bf16(g[ob][8 * kk + 2 * e], g[ob][8 * kk + 2 * e + 1], first, second);
            hi[ob][e] = first;
            lo[ob][e] = second;
          }
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb) {
          const uint32_t at = o.y[nb % o.NY] + base + (nb / o.NY) * 128 + 16 * kk * T::RB;
          const s16x4 b[2] = {lds_tr4(at), lds_tr4(at + 8 * T::RB)};
          const u32x4 bw = __builtin_bit_cast(u32x4, b);
#pragma unroll
          for (int ob = 0; ob < OB; ++ob) acc[ob][nb] = LpMma<bf16>::run(hi[ob], bw, acc[ob][nb]);
#pragma unroll
          for (int ob = 0; ob < OB; ++ob) acc[ob][nb] = LpMma<bf16>::run(lo[ob], bw, acc[ob][nb]);
        }
      }
    } else {
      u32x4 part[OB][2];
#pragma unroll 1
      for (int t = 0; t < TERMS; ++t) {
        term(part);
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            g[ob][2 * e] -= lo_f32(part[ob][e / 4][e % 4]);
            g[ob][2 * e + 1] -= hi_f32(part[ob][e / 4][e % 4]);
          }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int nb = 0; nb < D / 32; ++nb) {
        const float b = lds_at<float>(o.y[v & 3] + base + 8 * (v >> 2) * T::RB + nb * 128);
#pragma unroll
        for (int ob = 0; ob < OB; ++ob) acc[ob][nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(g[ob][v], b, acc[ob][nb], 0, 0, 0);
      }
  }
}

// NWO waves along the owners x NWS waves along a tile's rows; OB blocks of 32 owners per wave.
// A position's own item is left out of the sums (its logit becomes one that weighs nothing), and its weight g in LP_DX
// and LP_DY is the whole of it, g (1 - p) and the entropy's, formed before: as one of the sum's terms, p would round
// what the others add by 2^-24 each time, and where it is near 1 nothing else is left of 1 - p.  Few blocks hold an own
// item, so what costs is the question (a comparison of ids per block).
template <class E, int D, int OB, int NWO, int NWS, int MODE, bool ENT, int TERMS, int MINW>
__global__ __launch_bounds__(64 * NWO * NWS, MINW) void k_lp_sweep(LpArgs a) {
  using T = LpTile<E, D, NWS>;
  using L = TileReads<E, D>;
  constexpr int TI = T::TI, RB = T::RB, CPR = T::CPR, NT = 64 * NWO * NWS;
  constexpr int KC = L::KC;
  constexpr int PT = T::BYTES / 16 / NT;   // chunks a thread copies per tile
  constexpr bool ACC = MODE != LP_LSE, LSE = MODE == LP_LSE || MODE == LP_LSEO, DY = MODE == LP_DY;
  static_assert(T::BYTES % (16 * NT) == 0 && TI <= NT, "whole chunks per thread");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id(), h = l >> 5, r = l & 31;
  const int wo = w % NWO, ws = w / NWO;   // in scalar registers, and so is what follows from them
  // row numbers in 32 bits without a sign: at most 2^31 - 1 rows and a tile
  const uint32_t n_own = a.parts.owners(), n_str = a.parts.streamed();
  const SweepWork work = a.parts.work();
  const uint32_t ntiles = work.nt;

  L lo;
  lo.init();
  uint32_t o0 = 0, tb = 0, te = 0;   // the wave's first owner, the run's tiles of its block
  u32x4 bown[OB][KC];
  uint32_t oid[OB];                            // the owners' own items (not LP_DY)
  float olse[OB], oa[OB], obt[OB], og[OB];     // LP_DX: the owners' constants
  auto load_owners = [&]() {
    const uint32_t rr = settled(r), hh = settled(h);
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      const uint32_t o = min(o0 + 32 * ob + rr, n_own - 1);
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.own) + (int64_t)o * RB) + hh;
#pragma unroll
      for (int t = 0; t < KC; ++t) bown[ob][t] = p[2 * t];
      if constexpr (!DY) oid[ob] = (uint32_t)a.idc[o];
      if constexpr (MODE == LP_DX) {
        const LpRow c = a.rows[o];
        olse[ob] = c.lse2;
        oa[ob] = c.a;
        obt[ob] = c.b;
        og[ob] = c.g;
      }
    }
  };
  // the values of own items in the block of rows that begins at q0 become f(ob) (not LP_DY)
  auto own_items = [&](f32x16 (&x)[OB], uint32_t q0, auto f) {
    bool near = false;
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) near = near || oid[ob] - q0 < 32u;
    if (!ballot(near)) return;
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      const uint32_t at = oid[ob] - q0 - 4 * h;
#pragma unroll
      for (int v = 0; v < 16; ++v)
        x[ob][v] = at == (uint32_t)lp_row(v) ? f(ob) : x[ob][v];
    }
  };
  float m[OB], z[OB], tt[OB];   // LP_LSE(O): reference and sums
  f32x16 acc[ACC ? OB : 1][D / 32];
  constexpr bool LO = sizeof(E) == 4;
  const LpScale c2 = a.c2;
  // a logit that weighs nothing, finite after the factor c2
  const float far = fmaxf(-1e30f / c2.hi, -3e38f);

  // behind the two tile buffers (LP_DY): the rows' constants, [2][5][TI] words: lse2, a, b, g, id
  constexpr int PB = 5 * TI * 4;
  const uint32_t par0 = lds0 + 2 * T::BYTES;
  u32x4 nxt[PT];
  u32x4 nrow = u32x4{0u, 0u, 0u, 0u};
  uint32_t nid = 0;
  // Chunk q NT + tid of a tile: row q (NT / CPR) + tid / CPR.  One lane offset serves all q, beside
  // scalar ones; the swizzle repeats every 8 rows.
  constexpr int RPQ = NT / CPR;
  static_assert(RPQ % 8 == 0 || RPQ == 4, "rows per copy step");
  const uint32_t crow = tid / CPR, ccol = tid % CPR;
  const uint32_t st0 = crow * RB + ((ccol ^ (crow & T::SWM)) << 4), st1 = RPQ == 4 ? st0 ^ 64u : st0;
  auto fetch = [&](uint32_t t) {
    const char* src = static_cast<const char*>(a.str) + (int64_t)t * T::BYTES;
    if ((t + 1) * TI <= n_str) {
#pragma unroll
      for (int q = 0; q < PT; ++q) nxt[q] = *reinterpret_cast<const u32x4*>(src + q * (NT * 16) + (uint32_t)tid * 16);
    } else {   // rows beyond the end repeat the last one
      const uint32_t last = n_str - t * TI - 1;
#pragma unroll
      for (int q = 0; q < PT; ++q) nxt[q] = *reinterpret_cast<const u32x4*>(src + (min(crow + q * RPQ, last) * RB + ccol * 16));
    }
    if constexpr (DY) {
      if (tid < TI) {   // packed rows are padded with rows of no weight to whole tiles
        nrow = *reinterpret_cast<const u32x4*>(a.rows + ((int64_t)t * TI + tid));
        nid = (uint32_t)a.idc[(int64_t)t * TI + tid];
      }
    }
  };
  auto stash = [&](uint32_t t) {
    const uint32_t buf = lds0 + (t & 1) * T::BYTES;
#pragma unroll
    for (int q = 0; q < PT; ++q) lds_put(((q & 1) ? st1 : st0) + buf + q * (NT * 16), nxt[q]);
    if constexpr (DY) {
      if (tid < TI) {
        const uint32_t par = par0 + (t & 1) * PB + 4 * tid;
#pragma unroll
        for (int q = 0; q < 5; ++q) lds_put(par + q * TI * 4, q < 4 ? nrow[q < 4 ? q : 0] : nid);
      }
    }
  };

  // logits of 32 streamed rows (first one q0, at LDS offset base) against the wave's owners
  auto logits = [&](f32x16 (&x)[OB], uint32_t base, uint32_t q0) {
    const f32x16 zero = {};
    constexpr int KG = KC < LP_FRAGS ? KC : (D == 256 ? 2 : LP_FRAGS);   // fragments in flight
#pragma unroll
    for (int k0 = 0; k0 < KC; k0 += KG) {
      u32x4 f[KG];
#pragma unroll
      for (int k = 0; k < KG; ++k) f[k] = L::frag(lo, base, k0 + k);
#pragma unroll
      for (int k = 0; k < KG; ++k)
#pragma unroll
        for (int ob = 0; ob < OB; ++ob) x[ob] = LpMma<E>::run(f[k], bown[ob][k0 + k], k0 + k == 0 ? zero : x[ob]);
    }
    if constexpr (!DY) {
      if (q0 + 32 > n_str) {   // the last tile's rows beyond the end
        const int lim = (int)(n_str - q0) - 4 * h;
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (lp_row(v) >= lim) x[ob][v] = far;
      }
    }
    if constexpr (LSE) own_items(x, q0, [&](int) { return far; });
  };
  // m = max(m, the block's logits), the same in both lane halves of an owner
  auto raise = [&](f32x16 (&x)[OB]) {
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      float bm = m[ob];
#pragma unroll
      for (int v = 0; v < 16; ++v) bm = fmaxf(bm, x[ob][v] * c2.hi);
      m[ob] = fmaxf(bm, __shfl_xor(bm, 32));
    }
  };
  // the block's logits become weights, and join the sums
  auto weigh = [&](f32x16 (&x)[OB], uint32_t par, uint32_t q0) {
    if constexpr (LSE) {
#pragma unroll
      for (int ob = 0; ob < OB; ++ob) {
        float s = 0.0f, st = 0.0f;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float d = lp_less<LO>(x[ob][v], c2, m[ob]);
          x[ob][v] = exp2_fast(d);
          s += x[ob][v];
          if constexpr (ENT) st = fmaf(x[ob][v], d, st);
        }
        z[ob] += s;
        if constexpr (ENT) tt[ob] += st;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 pl, pa, pb;
        if constexpr (DY) {
          const uint32_t at = par + 32 * q + 16 * h;
          pl = lds_at<f32x4>(at);
          pa = lds_at<f32x4>(at + TI * 4);
          if constexpr (ENT) pb = lds_at<f32x4>(at + 2 * TI * 4);
        }
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = 4 * q + e;
            const float d = lp_less<LO>(x[ob][v], c2, DY ? pl[e] : olse[ob]);
            x[ob][v] = lp_weight<ENT>(d, DY ? pa[e] : oa[ob], DY ? pb[e] : obt[ob]);
          }
      }
      if constexpr (MODE == LP_DX) own_items(x, q0, [&](int ob) { return og[ob]; });
      if constexpr (DY) {
        if (ballot(lds_at<uint32_t>(par + 4 * TI * 4 + 4 * r) - o0 < 32 * OB)) {
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const uint32_t at = par + 4 * (lp_row(v) + 4 * h);
            const uint32_t id = lds_at<uint32_t>(at + 4 * TI * 4);
            const float g = lds_at<float>(at + 3 * TI * 4);
#pragma unroll
            for (int ob = 0; ob < OB; ++ob) x[ob][v] = id == o0 + 32 * ob + r ? g : x[ob][v];
          }
        }
      }
    }
  };
  constexpr int NB = TI / 32 / NWS;   // blocks of a tile per wave
  // All tiles of the split through f(LDS offset of the wave's first block, of its constants, its first row).
  auto sweep = [&](auto f) {
    fetch(tb);
    stash(tb);
#pragma unroll 1
    for (uint32_t t = tb; t < te; ++t) {
      __syncthreads();
      if (t + 1 < te) fetch(t + 1);
      f(lds0 + (t & 1) * T::BYTES + ws * (32 * RB), par0 + (t & 1) * PB + ws * 128, t * TI + ws * 32);
      if (t + 1 < te) stash(t + 1);
    }
    __syncthreads();   // the buffers may be filled again
  };
  auto main_tile = [&](uint32_t base, uint32_t par, uint32_t q0) {
#pragma unroll 1
    for (int i = 0; i < NB; ++i) {
      f32x16 x[OB];
      logits(x, base + i * (NWS * 32 * RB), q0 + i * NWS * 32);
      weigh(x, par + i * (NWS * 128), q0 + i * NWS * 32);
      if constexpr (ACC) lp_product<E, D, NWS, OB, TERMS>(acc, x, lo, base + i * (NWS * 32 * RB));
    }
  };
  auto run = [&]() {
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) m[ob] = LP_FLOOR;
    if constexpr (LSE) {
      // the largest logit of the wave's first block is the reference of the sums
      fetch(tb);
      stash(tb);
      __syncthreads();
      f32x16 x[OB];
      logits(x, lds0 + (tb & 1) * T::BYTES + ws * (32 * RB), tb * TI + ws * 32);
      raise(x);
      __syncthreads();
    }
#pragma unroll 1
    for (bool again = false;; again = true) {
      if constexpr (LSE) {
        if (again)   // true maxima of the run's tiles
          sweep([&](uint32_t base, uint32_t, uint32_t q0) {
#pragma unroll 1
            for (int i = 0; i < NB; ++i) {
              f32x16 x[OB];
              logits(x, base + i * (NWS * 32 * RB), q0 + i * NWS * 32);
              raise(x);
            }
          });
      }
#pragma unroll
      for (int ob = 0; ob < OB; ++ob) {
        z[ob] = tt[ob] = 0.0f;
        if constexpr (ACC)
#pragma unroll
          for (int nb = 0; nb < D / 32; ++nb)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[ob][nb][v] = 0.0f;
      }
      sweep(main_tile);
      if constexpr (!LSE) break;
      // exp2 has the range for logits up to 60 (base 2) beyond the reference; further (or with NaN among
      // them) the references become the true maxima and the sums are taken once more
      bool over = false;
#pragma unroll
      for (int ob = 0; ob < OB; ++ob) over = over || !(z[ob] < LP_REF_LIMIT);
      if (again || !__syncthreads_or(over)) break;
    }
  };

  const uint64_t u1 = min(work.total, (uint64_t)(blockIdx.x + 1) * work.per);
#pragma unroll 1
  for (uint64_t u = (uint64_t)blockIdx.x * work.per; u < u1; u += te - tb) {
    const uint32_t b = (uint32_t)div_u64(u, ntiles);
    tb = (uint32_t)(u - (uint64_t)b * ntiles);
    te = (uint32_t)min((uint64_t)ntiles, tb + (u1 - u));
    o0 = b * (32 * OB * NWO) + wo * (32 * OB);
    load_owners();
    run();
    // part [slot][ws][owner of the block]; settled(): the lanes' offsets are formed here, not
    // kept in registers through the sweep
    const int64_t part = (work.slot(b, blockIdx.x) * NWS + ws) * (32 * OB * NWO) + wo * (32 * OB);
    const int rr = settled(r), hh = settled(h);
    if constexpr (LSE) {
#pragma unroll
      for (int ob = 0; ob < OB; ++ob) {
        // the two lane halves hold different rows of the same owner, against one reference
        const float zz = z[ob] + __shfl_xor(z[ob], 32), t0 = tt[ob] + __shfl_xor(tt[ob], 32);
        if (hh == 0) {
          a.stat[part + 32 * ob + rr] = float4{m[ob], zz, ENT ? t0 : 0.0f, 0.0f};
        }
      }
    }
    if constexpr (ACC) {   // whole blocks: rows beyond the last owner hold values that nothing reads
      float* out = a.out + part * D;
      const uint32_t lane = 4 * hh * D + rr;
#pragma unroll
      for (int ob = 0; ob < OB; ++ob)
#pragma unroll
        for (int v = 0; v < 16; ++v)
#pragma unroll
          for (int nb = 0; nb < D / 32; ++nb) out[(32 * ob + lp_row(v)) * D + 32 * nb + lane] = acc[ob][nb][v];
    }
  }
}

// ------------------------------------------------------------------ packing
// (12 us for 51,200 ids of rows of 64 bf16, 25 MB; 6 us for 256.)
// Workgroup b takes ids [b per, (b + 1) per): it counts the ids before them that lie in
// [0, C) itself (an L2-resident read of 4 bytes a position, in place of a scan's further
// launches), then writes the list of its own, the packed rows and ids, and the (unscaled)
// logit of each row's own item, the diagonal of a 32 x 32 product.  The last workgroup fills the
// padding with zero rows.
constexpr int PACK_THREADS = 256;
constexpr int64_t PACK_BLOCKS = 256, PACK_LEAST = 64;   // workgroups at most, ids of each at least

template <class E, int D>
__global__ __launch_bounds__(PACK_THREADS) void k_lp_pack(const E* __restrict__ X, const E* __restrict__ Y,
                                                          const int32_t* __restrict__ ids, int64_t s, int64_t C,
                                                          int64_t per, int64_t pad, int32_t* __restrict__ nv,
                                                          int32_t* __restrict__ list, int32_t* __restrict__ inv,
                                                          E* __restrict__ Xc, int32_t* __restrict__ idc,
                                                          float* __restrict__ own) {
  constexpr int RB = D * (int)sizeof(E), KC = RB / 32, NW = PACK_THREADS / WAVE;
  __shared__ int32_t wsum[NW];
  __shared__ int32_t src[PACK_THREADS];
  const int tid = threadIdx.x, w = tid >> 6, l = lane_id(), h = l >> 5, r = l & 31;
  const int64_t i0 = (int64_t)blockIdx.x * per, i1 = min(s, i0 + per);
  auto good = [&](int64_t i, int64_t end) {
    const int id = i < end ? ids[i] : -1;
    return id >= 0 && id < C;
  };
  int before = 0;
  int64_t from = 0;
  if ((reinterpret_cast<uintptr_t>(ids) & 15) == 0) {
    const uint32_t last = (uint32_t)(C - 1);
#pragma unroll 8
    for (int64_t q = tid; q < i0 / 4; q += PACK_THREADS) {
      const u32x4 v = reinterpret_cast<const u32x4*>(ids)[q];
      before += (v[0] <= last) + (v[1] <= last) + (v[2] <= last) + (v[3] <= last);
    }
    from = i0 / 4 * 4;
  }
#pragma unroll 8
  for (int64_t i = from + tid; i < i0; i += PACK_THREADS) before += good(i, i0) ? 1 : 0;
  before = wave_sum(before);
  if (l == 0) wsum[w] = before;
  __syncthreads();
  int64_t done = 0;
#pragma unroll
  for (int q = 0; q < NW; ++q) done += wsum[q];
  for (int64_t b = i0; b < i1; b += PACK_THREADS) {
    const int64_t i = b + tid;
    const bool on = good(i, i1);
    const uint64_t mask = ballot(on);
    __syncthreads();   // wsum and src of the step before are read
    if (l == 0) wsum[w] = popc(mask);
    __syncthreads();
    int at = popc(mask & lanemask_lt()), tot = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      if (q < w) at += wsum[q];
      tot += wsum[q];
    }
    if (i < i1) inv[i] = on ? (int32_t)(done + at) : -1;
    if (on) {
      list[done + at] = (int32_t)i;
      src[at] = (int32_t)i;
    }
    __syncthreads();
    for (int q = w * 32; q < tot; q += NW * 32) {   // 32 rows per wave
      const int64_t pos = src[min(q + r, tot - 1)];
      const int32_t id = ids[pos];
      const u32x4* px = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(X) + pos * RB);
      const u32x4* py = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(Y) + (int64_t)id * RB);
      u32x4* pc = reinterpret_cast<u32x4*>(reinterpret_cast<char*>(Xc) + (done + q + r) * RB);
      f32x16 x = {};
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const u32x4 fx = px[2 * k + h], fy = py[2 * k + h];
        x = LpMma<E>::run(fy, fx, x);
        if (q + r < tot) pc[2 * k + h] = fx;
      }
      float d = 0.0f;
      bool mine = false;
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (lp_row(v) + 4 * h == r) {
          d = x[v];
          mine = true;
        }
      if (mine && q + r < tot) {
        own[done + q + r] = d;
        idc[done + q + r] = id;
      }
    }
    done += tot;
  }
  if (blockIdx.x + 1 == gridDim.x) {
    const int64_t end = min(pad, (done + LP_ROW_PAD - 1) / LP_ROW_PAD * LP_ROW_PAD);
    for (int64_t q = done * (RB / 16) + tid; q < end * (RB / 16); q += PACK_THREADS)
      reinterpret_cast<u32x4*>(Xc)[q] = u32x4{0u, 0u, 0u, 0u};
    for (int64_t q = done + tid; q < pad; q += PACK_THREADS) idc[q] = -1;
    if (tid == 0) *nv = (int32_t)done;
  }
}

// ------------------------------------------------------------------ joins
// L lanes per position (1, a wave, a workgroup): the parts of the others' sum -> log-sum-exp, log-probability, entropy.
// Where the own item is most of it, log p = -log1p(the others' sum over the own term), which keeps every digit of 1 - p.
constexpr int FINISH_WIDE = 1024;
template <int L>
__global__ __launch_bounds__(L > WAVE ? L : 256) void k_lp_finish(
    const int32_t* __restrict__ inv, int64_t s, SweepParts parts, const float4* __restrict__ stat,
    const float* __restrict__ own, LpScale c2, float2* __restrict__ lse2, float* __restrict__ logp_c, float* __restrict__ ent_c,
    float* __restrict__ logp, float* __restrict__ entropy) {
  constexpr int NT = L > WAVE ? L : 256, UNR = 4;
  const int64_t i = ((int64_t)blockIdx.x * NT + threadIdx.x) / L;
  const int l = threadIdx.x % L;
  if (i >= s) return;
  const int64_t r = inv[i];
  if (r < 0) {
    if (l == 0) {
      logp[i] = 0.0f;
      if (entropy) entropy[i] = 0.0f;
    }
    return;
  }
  const SweepWork w = parts.work();
  const uint32_t b = (uint32_t)r / parts.block, in = (uint32_t)r % parts.block;
  const int64_t p0 = w.slot(b, w.first(b)) * parts.nws, p1 = (w.slot(b, w.last(b)) + 1) * parts.nws;
  float mm = NEG_INF, zz = 0.0f, tt = 0.0f;
  auto add = [&](float mp, float zp, float tp) {   // mp = NEG_INF: nothing
    const float mn = fmaxf(mm, mp);
    const float f0 = mm == NEG_INF ? 0.0f : exp2_fast(mm - mn), f1 = mp == NEG_INF ? 0.0f : exp2_fast(mp - mn);
    tt = (mm == NEG_INF ? 0.0f : (tt + zz * (mm - mn)) * f0) + (mp == NEG_INF ? 0.0f : (tp + zp * (mp - mn)) * f1);
    zz = zz * f0 + zp * f1;
    mm = mn;
  };
  for (int64_t p = p0 + l; p < p1; p += UNR * L) {
    float4 x[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      x[u] = stat[min(p + u * L, p1 - 1) * parts.block + in];
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u)
      if (p + u * L < p1) add(x[u].x, x[u].y, x[u].z);
  }
  if constexpr (L > 1) {
    auto join = [&]() {
      const float mn = wave_max(mm);
      const float f = mm == NEG_INF ? 0.0f : exp2_fast(mm - mn);
      tt = wave_sumf(mm == NEG_INF ? 0.0f : (tt + zz * (mm - mn)) * f);
      zz = wave_sumf(zz * f);
      mm = mn;
    };
    join();
    if constexpr (L > WAVE) {
      __shared__ float sm[L / WAVE], sz[L / WAVE], st[L / WAVE];
      if (lane_id() == 0) {
        sm[l / WAVE] = mm;
        sz[l / WAVE] = zz;
        st[l / WAVE] = tt;
      }
      __syncthreads();
      if (l >= WAVE) return;
      const bool one = l < L / WAVE;
      mm = one ? sm[l] : NEG_INF;
      zz = one ? sz[l] : 0.0f;
      tt = one ? st[l] : 0.0f;
      join();
    }
    if (l != 0) return;
  }
  // the own logit in two floats; the others' sum zz stands for zz 2^mm
  const float o = own[r], x2 = o * c2.hi, x2lo = fmaf(o, c2.lo, fmaf(o, c2.hi, -x2));
  // over the own term (NaN stays); x2lo is below a step of x2, so it goes in as a factor
  const float t1 = zz * exp2_fast(fminf(mm - x2, 64.0f)) * fmaf(-LN2, x2lo, 1.0f);
  const bool mostly = t1 < 1.0f;
  const float e = mostly ? 0.0f : exp2_fast(x2 - mm), all = zz + e;   // at most zz, where it is taken
  // log-sum-exp as two floats: a step of one alone, 2^-20 for sums beyond 2^16, is as large as the rest
  const float base = mostly ? x2 : mm, more = mostly ? log1pf(t1) * (1.0f / LN2) : log2f(all);
  const float l2 = base + more, back = l2 - base;
  const float rest = (base - (l2 - back)) + (more - back) + (mostly ? x2lo : 0.0f);
  const float lp = mostly ? -log1pf(t1) : (lp_less<true>(o, c2, l2) - rest) * LN2;
  lse2[r] = float2{l2, rest};
  logp_c[r] = lp;
  logp[i] = lp;
  if (entropy) {
    // sum of p (lse - x), the own item's part apart where it is most: (1 - p) times the others' mean distance, and p log p
    float H;
    if (mostly) {
      const float p = 1.0f / (1.0f + t1);
      H = zz > 0.0f ? t1 * p * ((l2 - mm) - tt / zz) * LN2 - p * lp : 0.0f;
    } else {
      H = (more - (tt + e * (x2 - mm)) / all) * LN2;
    }
    entropy[i] = H;
    ent_c[r] = H;
  }
}

// Constants of the gradient per packed row; rows of no weight up to the padding.  What lse2's second float leaves goes
// into the factors.
template <bool ENT>
__global__ __launch_bounds__(256) void k_lp_coef(const int32_t* __restrict__ nv_p, const int32_t* __restrict__ list,
                                                 int64_t pad, const float2* __restrict__ lse2,
                                                 const float* __restrict__ logp_c, const float* __restrict__ ent_c,
                                                 const float* __restrict__ dlogp, const float* __restrict__ dent,
                                                 float inv_t, LpRow* __restrict__ rows) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= pad) return;
  LpRow c{LP_NEVER, 0.0f, 0.0f, 0.0f};
  if (r < *nv_p) {
    const int64_t i = list[r];
    const float g = dlogp[i] * inv_t, h = ENT ? dent[i] * inv_t : 0.0f;
    const float2 l2 = lse2[r];
    const float lp = logp_c[r], H = ENT ? ent_c[r] : 0.0f, f = fmaf(-LN2, l2.y, 1.0f);
    c.lse2 = l2.x;
    c.a = (ENT ? fmaf(h, H, g) : g) * f;
    c.b = h * LN2 * f;
    c.g = g * -expm1f(lp);
    if constexpr (ENT) c.g -= expf(lp) * h * (lp + H);
  }
  rows[r] = c;
}

__device__ __forceinline__ void put4(void* out, int64_t at, float4 v, bool b16) {
  if (b16) {
    uint2 o;
    o.x = pack_bf16(v.x, v.y);
    o.y = pack_bf16(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = o;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  }
}

// d / 4 lanes hold a row's columns, `groups` of those share its parts: 1, or a wave's worth (256 / d, at least 1)
// where a row has 16 parts or more, so that many loads are in flight.  (256 positions, 33 parts of 64 floats each:
// 12 -> 5 us with 4 groups; 51,200 positions, 3 to 4 parts: 14 -> 35 us.)  Sums in a fixed order.
struct JoinLane {
  int64_t row;
  int col, group, groups;
  __device__ __forceinline__ JoinLane(int d, int n) : groups(n) {
    const int per = d / 4, rest = (int)threadIdx.x % per;
    const int64_t unit = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x) / per;
    row = unit / groups;
    group = (int)(unit % groups);
    col = rest * 4;
  }
  // the groups' sums, in every lane
  __device__ __forceinline__ void sum(float4& v, int d) const {
    for (int o = d / 4; o < d / 4 * groups; o *= 2)
      v = float4{v.x + __shfl_xor(v.x, o), v.y + __shfl_xor(v.y, o), v.z + __shfl_xor(v.z, o), v.w + __shfl_xor(v.w, o)};
  }
};
int join_groups(const SweepParts& p, int d) {
  const int64_t nb = (p.n_own + p.block - 1) / p.block;
  return !p.whole && (int64_t)p.grid * p.nws >= 16 * nb ? std::max(1, 256 / d) : 1;
}
dim3 join_grid(int64_t n, int d, int groups) {   // at most 2^31 threads along x
  const int64_t blocks = (n * (d / 4) * groups + 255) / 256, x = std::min<int64_t>(blocks, 1 << 23);
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

// out row = sum of the parts' rows.  inv (dX): the row of the parts for each output row (or -1: zeros).
__global__ __launch_bounds__(256) void k_lp_join(SweepParts parts, int d, int groups, const int32_t* __restrict__ inv, int64_t n,
                                                 void* __restrict__ out, int b16) {
  const JoinLane q(d, groups);
  if (q.row >= n) return;   // a row's lanes together
  const int64_t i = q.row;
  const int c = q.col;
  const int64_t r = inv ? inv[i] : i;
  float4 v = float4{0.0f, 0.0f, 0.0f, 0.0f};
  if (r >= 0) {
    parts.each(parts.work(), r, [&](int64_t at) {
      const float4 w = *reinterpret_cast<const float4*>(parts.rows + at * d + c);
      v = float4{v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w};
    }, q.group, q.groups);
    q.sum(v, d);
  }
  if (q.group == 0) put4(out, i * d + c, v, b16 != 0);
}

// dX without an entropy gradient, from the forward pass's sums O of 2^(x2 - m) y_j over the other items:
//   dX_i = g_i ((1 - p_own) y_own - sum over the parts of O 2^(m - lse2))
template <class E>
__global__ __launch_bounds__(256) void k_lp_dx(SweepParts parts, const float4* __restrict__ stat, int d, int groups,
                                               const int32_t* __restrict__ inv, int64_t s, const E* __restrict__ Y,
                                               const int32_t* __restrict__ idc, const float2* __restrict__ lse2,
                                               const float* __restrict__ logp_c, const float* __restrict__ dlogp,
                                               float inv_t, void* __restrict__ out, int b16) {
  const JoinLane q(d, groups);
  if (q.row >= s) return;   // a row's lanes together
  const int64_t i = q.row;
  const int c = q.col;
  const int64_t r = inv[i];
  float4 v = float4{0.0f, 0.0f, 0.0f, 0.0f};
  if (r >= 0) {
    const float2 l2 = lse2[r];
    const float g = dlogp[i] * inv_t, rest = -expm1f(logp_c[r]);
    const E* yp = Y + (int64_t)idc[r] * d + c;
    const float4 y = float4{to_f32(yp[0]), to_f32(yp[1]), to_f32(yp[2]), to_f32(yp[3])};
    parts.each(parts.work(), r, [&](int64_t at) {
      const float f = exp2_fast((stat[at].x - l2.x) - l2.y);
      const float4 x = *reinterpret_cast<const float4*>(parts.rows + at * d + c);
      v = float4{fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w)};
    }, q.group, q.groups);
    q.sum(v, d);
    v = float4{g * fmaf(rest, y.x, -v.x), g * fmaf(rest, y.y, -v.y), g * fmaf(rest, y.z, -v.z), g * fmaf(rest, y.w, -v.w)};
  }
  if (q.group == 0) put4(out, i * d + c, v, b16 != 0);
}

// ------------------------------------------------------------------ host side
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int LP_CUS = 256;

// Launch shapes, by the bytes of a row: OB blocks of 32 owners per wave (more: fewer LDS reads per product; fewer:
// more waves per SIMD to overlap the exponentials with the products), MW waves per SIMD (the registers allow
// them; the grid fills the card once), NWO waves per workgroup.  Whole calls with bf16 gradients, without / with
// entropies, us (spills: words per lane that do not fit into registers):
//   D 64, 51,200 x 30,000:   OB 2 MW 2  933 / 1,222;  OB 1 MW 3  997 / 1,281;  OB 1 MW 4  1,031 / 1,286
//   D 128, 8,192 x 30,000:   OB 1 MW 2  369 / 454;  OB 1 MW 3  388 / 470;  OB 2 MW 1  394 / 485 (with float32 gradients
//                            501 / 579, 545 / 596 and 511 / 573)
//   D 256, 4,099 x 50,021:   NWO 8  588 / 748;  NWO 4  672 / 1,028;  NWO 8 MW 1  975 / 1,165
//   LP_LSE, MW 3 against 2:  D 128, 2,047 x 200,000  132 / 137;  D 256, 4,099 x 50,021  120 / 128
// Spills remain at D 256 (LP_LSEO 10 to 27, LP_DX 14 to 22, LP_DY 35 to 60; float32 24, 0 and 51 to 74), in the few-
// positions LP_LSEO at D 128 (3 to 21) and in LP_LSE at D 128 (6 to 8).
// A second block's logits in flight while the first is weighed gave LP_DY at D 64 less than 1 %, and is not done.
// Up to 32 OB positions the waves of a workgroup share their owners and split each tile's rows instead (NWS 4;
// a block of owners that is mostly empty costs as much as a full one): 5 x 1,000,000, LP_LSE 25 against 62.
template <class E, int D> struct LpShape {
  static constexpr bool B = sizeof(E) == 2;
  static constexpr int OB_LSE = B && D <= 128 ? 2 : 1;
  static constexpr int MW_LSE = B ? 3 : (D <= 128 ? 3 : 2);
  static constexpr int OB_GRAD = B && D <= 64 ? 2 : 1;
  static constexpr int MW_GRAD = !B && D > 64 ? 1 : 2;
  static constexpr int NWO_GRAD = B && D == 256 ? 8 : 4;
  static constexpr int NWS_FEW = D * (int)sizeof(E) <= 256 ? 4 : 1;
  static constexpr int MW_FEW = D * (int)sizeof(E) <= 128 ? 3 : 2;
};

struct LpSweep {   // one sweep's shape
  int ob, nwo, nws, ti;
  uint32_t grid;
  bool whole;
  int64_t slots(int64_t n_own) const { return (ceil_div(n_own, block()) + (whole ? 0 : grid)) * nws; }   // parts of a block each
  int64_t block() const { return 32 * (int64_t)ob * nwo; }
};

template <class E, int D>
LpSweep lp_shape(int mode, int64_t n_own, int64_t n_str) {
  using S = LpShape<E, D>;
  LpSweep p{};
  p.ob = mode == LP_LSE ? S::OB_LSE : S::OB_GRAD;
  const bool few = mode != LP_DY && S::NWS_FEW > 1 && n_own <= 32 * p.ob;
  p.nwo = few ? 1 : mode == LP_LSE ? 4 : S::NWO_GRAD;
  p.nws = few ? S::NWS_FEW : 1;
  p.ti = few ? LpTile<E, D, S::NWS_FEW>::TI : LpTile<E, D, 1>::TI;
  const int64_t units = ceil_div(n_own, p.block()) * ceil_div(n_str, p.ti);
  int waves = mode == LP_LSE ? S::MW_LSE : S::MW_GRAD;   // per SIMD
  if (few) waves = std::min<int>(waves, S::MW_FEW);
  p.grid = (uint32_t)std::min<int64_t>(LP_CUS * waves * 4 / (p.nwo * p.nws), units);
  // items as owners (their number is known here): whole blocks where that leaves at most 1/16 of the grid's work idle
  const int64_t nb = ceil_div(n_own, p.block());
  p.whole = mode == LP_DY && (ceil_div(nb, p.grid) * p.grid - nb) * 16 <= nb;
  return p;
}

struct LpLayout {
  int64_t pad;
  size_t nv, list, inv, idc, own, lse2, logp, ent, rows, xc, stat, o, dx, bytes;
};

template <class E, int D>
LpLayout lp_layout_t(int64_t s, int64_t C, uint32_t flags) {
  const bool grad = !(flags & RECE_FLAG_NO_GRAD), ent = flags & RECE_FLAG_ENTROPY;
  LpLayout y{};
  y.pad = ceil_div(s, LP_ROW_PAD) * LP_ROW_PAD;
  // without entropies the forward pass of a gradient takes the sums of item rows along
  const bool fused = grad && !ent;
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
  y.own = take(y.pad * 4);
  y.lse2 = take(y.pad * 8);
  y.logp = take(y.pad * 4);
  y.ent = take(ent ? y.pad * 4 : 0);
  y.xc = take((size_t)y.pad * D * sizeof(E));
  const LpSweep f = lp_shape<E, D>(fused ? LP_LSEO : LP_LSE, s, C);
  const size_t parts = (size_t)f.slots(s) * f.block() * 4;
  size_t base = off;
  y.stat = take(parts * 4);
  if (fused) {
    y.o = take(parts * D);
    base = off;
  }
  const size_t fwd = off;
  off = base;
  if (grad) {
    const LpSweep x = lp_shape<E, D>(LP_DX, s, C), v = lp_shape<E, D>(LP_DY, C, s);
    y.rows = take(y.pad * sizeof(LpRow));
    // dX is finished before the dY sweep starts
    y.dx = take(std::max(ent ? (size_t)x.slots(s) * x.block() : 0, (size_t)v.slots(C) * v.block()) * D * 4);
  }
  y.bytes = std::max(fwd, off);
  return y;
}

template <class E, int D, int OB, int NWO, int NWS, int MODE, bool ENT, int TERMS, int MINW>
hipError_t lp_launch_t(const LpArgs& a, hipStream_t st) {
  using T = LpTile<E, D, NWS>;
  const size_t lds = 2 * (size_t)T::BYTES + (MODE == LP_DY ? 2 * T::TI * (sizeof(LpRow) + 4) : 0);
  auto kern = k_lp_sweep<E, D, OB, NWO, NWS, MODE, ENT, TERMS, MINW>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(a.parts.grid), dim3(64 * NWO * NWS), lds, st, a);
  return hipGetLastError();
}

template <class E, int D, int MODE, bool ENT>
hipError_t lp_launch(const LpArgs& a, hipStream_t st) {
  using S = LpShape<E, D>;
  constexpr int NWO = MODE == LP_LSE ? 4 : S::NWO_GRAD;
  constexpr int OB = MODE == LP_LSE ? S::OB_LSE : S::OB_GRAD, MINW = MODE == LP_LSE ? S::MW_LSE : S::MW_GRAD;
  constexpr bool THREE = sizeof(E) == 2 && MODE != LP_LSE;   // has a variant of three terms
  constexpr int TERMS = THREE ? 2 : 1;
  if constexpr (MODE != LP_DY && S::NWS_FEW > 1) {
    constexpr int FEW = MINW < S::MW_FEW ? MINW : S::MW_FEW;
    if (a.parts.nws > 1) {
      if constexpr (THREE)
        if (a.terms == 3) return lp_launch_t<E, D, OB, 1, S::NWS_FEW, MODE, ENT, 3, FEW>(a, st);
      return lp_launch_t<E, D, OB, 1, S::NWS_FEW, MODE, ENT, TERMS, FEW>(a, st);
    }
  }
  if constexpr (THREE)
    if (a.terms == 3) return lp_launch_t<E, D, OB, NWO, 1, MODE, ENT, 3, MINW>(a, st);
  return lp_launch_t<E, D, OB, NWO, 1, MODE, ENT, TERMS, MINW>(a, st);
}

// Float32 results take all 24 bits of a weight, bf16 results two bf16 terms: 2^-16 of a weight is 1/256 of the
// result's own rounding.  (One term, 2^-8, would show in results that are small against their weights' sum.)
template <class E> int lp_terms(uint32_t flags) { return sizeof(E) == 4 ? 1 : flags & RECE_FLAG_BF16_GRADS ? 2 : 3; }

#define LP_TRY(call)                     \
  do {                                   \
    const hipError_t e_ = (call);        \
    if (e_ != hipSuccess) return e_;     \
  } while (0)

template <class E>
LpScale lp_scale(float temperature) {
  const double c = 1.4426950408889634 / (double)temperature;
  LpScale s{(float)c, 0.0f};
  if (sizeof(E) == 4 && std::isfinite(s.hi)) s.lo = (float)(c - (double)s.hi);
  return s;
}

template <class T> T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

template <class E, int D>
SweepParts lp_parts(int mode, int64_t n_own, int64_t n_str, const int32_t* nv, const float* rows) {
  const LpSweep f = lp_shape<E, D>(mode, n_own, n_str);
  SweepParts p{};
  p.nv = nv;
  p.n_own = n_own;
  p.n_str = n_str;
  p.own_is_pos = mode != LP_DY;
  p.block = (uint32_t)f.block();
  p.tile = (uint32_t)f.ti;
  p.grid = f.grid;
  p.nws = f.nws;
  p.whole = f.whole;
  p.rows = rows;
  return p;
}

template <class E, int D>
hipError_t lp_forward_t(int64_t s, int64_t C, float temperature, uint32_t flags, const void* X, const void* Y,
                        const int32_t* ids, void* ws, float* logp, float* entropy, hipStream_t st) {
  const LpLayout y = lp_layout_t<E, D>(s, C, flags);
  const LpScale c2 = lp_scale<E>(temperature);
  const int64_t per = std::max<int64_t>(PACK_LEAST, ceil_div(s, PACK_BLOCKS));
  hipLaunchKernelGGL((k_lp_pack<E, D>), dim3((unsigned)ceil_div(s, per)), dim3(PACK_THREADS), 0, st,
                     static_cast<const E*>(X), static_cast<const E*>(Y), ids, s, C, per, y.pad, at<int32_t>(ws, y.nv),
                     at<int32_t>(ws, y.list), at<int32_t>(ws, y.inv), at<E>(ws, y.xc), at<int32_t>(ws, y.idc),
                     at<float>(ws, y.own));
  LP_TRY(hipGetLastError());
  const bool fused = !entropy && !(flags & RECE_FLAG_NO_GRAD);
  LpArgs a{};
  a.own = at<E>(ws, y.xc);
  a.str = Y;
  a.parts = lp_parts<E, D>(fused ? LP_LSEO : LP_LSE, s, C, at<int32_t>(ws, y.nv), nullptr);
  a.c2 = c2;
  a.stat = at<float4>(ws, y.stat);
  a.idc = at<int32_t>(ws, y.idc);
  a.out = at<float>(ws, y.o);
  a.terms = lp_terms<E>(flags);
  if (fused)
    LP_TRY((lp_launch<E, D, LP_LSEO, false>(a, st)));
  else if (entropy)
    LP_TRY((lp_launch<E, D, LP_LSE, true>(a, st)));
  else
    LP_TRY((lp_launch<E, D, LP_LSE, false>(a, st)));
  // few positions have many parts each: a workgroup for each while the card holds them at once, or a wave; many have few
  const int lanes = s <= LP_CUS ? FINISH_WIDE : s <= 8192 ? WAVE : 1, threads = std::max(256, lanes);
  auto finish = lanes == FINISH_WIDE ? k_lp_finish<FINISH_WIDE> : lanes == WAVE ? k_lp_finish<WAVE> : k_lp_finish<1>;
  hipLaunchKernelGGL(finish, dim3((unsigned)ceil_div(s * lanes, threads)), dim3(threads), 0, st, at<int32_t>(ws, y.inv), s,
                     a.parts, a.stat, at<float>(ws, y.own), c2, at<float2>(ws, y.lse2), at<float>(ws, y.logp), at<float>(ws, y.ent), logp,
                     entropy);
  return hipGetLastError();
}

template <class E, int D>
hipError_t lp_backward_t(int64_t s, int64_t C, float temperature, uint32_t flags, const void* Y, void* ws,
                         const float* dlogp, const float* dent, void* dX, void* dY, hipStream_t st) {
  const LpLayout y = lp_layout_t<E, D>(s, C, flags);
  const float inv_t = 1.0f / temperature;
  const LpScale c2 = lp_scale<E>(temperature);
  const int b16 = flags & RECE_FLAG_BF16_GRADS ? 1 : 0, terms = lp_terms<E>(flags);
  const int32_t* nv = at<int32_t>(ws, y.nv);
  auto coef = dent ? k_lp_coef<true> : k_lp_coef<false>;
  hipLaunchKernelGGL(coef, dim3((unsigned)ceil_div(y.pad, 256)), dim3(256), 0, st, nv, at<int32_t>(ws, y.list), y.pad,
                     at<float2>(ws, y.lse2), at<float>(ws, y.logp), at<float>(ws, y.ent), dlogp, dent, inv_t,
                     at<LpRow>(ws, y.rows));
  LP_TRY(hipGetLastError());
  LpArgs a{};
  a.c2 = c2;
  a.rows = at<LpRow>(ws, y.rows);
  a.terms = terms;
  a.idc = at<int32_t>(ws, y.idc);
  auto join = [&](const int32_t* inv, int64_t n, void* out) {
    const int groups = join_groups(a.parts, D);
    hipLaunchKernelGGL(k_lp_join, join_grid(n, D, groups), dim3(256), 0, st, a.parts, D, groups, inv, n, out, b16);
    return hipGetLastError();
  };
  if (flags & RECE_FLAG_ENTROPY) {
    a.own = at<E>(ws, y.xc);
    a.str = Y;
    a.out = at<float>(ws, y.dx);
    a.parts = lp_parts<E, D>(LP_DX, s, C, nv, a.out);
    if (dent)
      LP_TRY((lp_launch<E, D, LP_DX, true>(a, st)));
    else
      LP_TRY((lp_launch<E, D, LP_DX, false>(a, st)));
    LP_TRY(join(at<int32_t>(ws, y.inv), s, dX));
  } else {
    const SweepParts sums = lp_parts<E, D>(LP_LSEO, s, C, nv, at<float>(ws, y.o));
    const int groups = join_groups(sums, D);
    hipLaunchKernelGGL((k_lp_dx<E>), join_grid(s, D, groups), dim3(256), 0, st, sums,
                       at<float4>(ws, y.stat), D, groups,
                       at<int32_t>(ws, y.inv), s, static_cast<const E*>(Y), a.idc, at<float2>(ws, y.lse2),
                       at<float>(ws, y.logp), dlogp, inv_t, dX, b16);
    LP_TRY(hipGetLastError());
  }
  a.own = Y;
  a.str = at<E>(ws, y.xc);
  a.out = at<float>(ws, y.dx);
  a.parts = lp_parts<E, D>(LP_DY, C, s, nv, a.out);
  if (dent)
    LP_TRY((lp_launch<E, D, LP_DY, true>(a, st)));
  else
    LP_TRY((lp_launch<E, D, LP_DY, false>(a, st)));
  return join(nullptr, C, dY);
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
