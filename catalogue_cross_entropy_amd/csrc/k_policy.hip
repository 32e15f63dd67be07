// Losses on log-probabilities of ragged sequences, with their gradients in the same pass:
// the clipped policy loss with a KL and an entropy term, and the preference loss over
// groups of sequences.  Formulas in include/rece.h.  Both are bound by memory: a token is
// a few floats read and one written, and every token is touched once (the policy loss
// reads the mask a second time, for the number of tokens its mean divides by).
// Sums and the weights of a mean are float64, token by token: a float32 sum over millions of tokens would lose the
// small differences these losses are made of, and one weight rounded to float32 would be off for all tokens alike.
//
// Measured (MI355X), calls back to back:
//   policy, 4.2M tokens float32 in 8,192 sequences, KL, mask: mean over tokens 36 us (75 MB; the tile kernel 29.5 us,
//     2.5 TB/s: one generation of workgroups, vector unit 40 % busy, waves waiting 56 % of their cycles), over
//     sequences 41 us of kernels in a graph, 49 a call (four launches)
//   policy, 16 sequences of 24 tokens: 9 us in one workgroup, of a call of 16 us (the call bounds it)
//   preference, 3.3M tokens bf16 in 2,048 groups of up to 8, softmax: 27 us (23 MB; loads one after the other:
//     offsets, tokens, the group's float64 terms, the gradient; vector unit 30 % busy, waves waiting 70 %)
//   preference, 131,072 pairs of items: 24 us, 16 of them the mean of the groups' losses by one workgroup
//   preference, 256 pairs of items: 7 us, of a call of 17.5 us
#include <algorithm>
#include <cmath>

#include "rece_device.h"
#include "rece_ops.h"

namespace rece {

namespace {

__device__ __forceinline__ uint32_t bf16_of(float x) { return x != x ? 0x7FC0u : bf16_bits_rne(x); }
__device__ __forceinline__ void put(float* p, int64_t t, float v) { p[t] = v; }
__device__ __forceinline__ void put(bf16* p, int64_t t, float v) { p[t].bits = (uint16_t)bf16_of(v); }

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = WAVE / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double wave_max_d(double v) {
#pragma unroll
  for (int o = WAVE / 2; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}

// Sum of v over the workgroup in a fixed order, in every thread.  sh: one double per wave;
// all threads call it, and it can be called again at once.
template <int NT>
__device__ __forceinline__ double block_sum_d(double v, double* sh) {
  v = wave_sum_d(v);
  __syncthreads();
  if (lane_id() == 0) sh[threadIdx.x / WAVE] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < NT / WAVE; ++w) s += sh[w];
  return s;
}

// offsets[i] inside [0, n].
__device__ __forceinline__ int64_t offset_at(const int32_t* __restrict__ offs, int64_t i, int64_t n) {
  return min(max((int64_t)offs[i], (int64_t)0), n);
}

// Sequence of token t among lo .. hi (inclusive): the last i with offsets[i] <= t, or lo.
__device__ __forceinline__ int64_t seq_of(const int32_t* __restrict__ offs, int64_t lo, int64_t hi, int64_t t) {
  while (lo < hi) {
    const int64_t m = (lo + hi + 1) / 2;
    if (offs[m] <= t) lo = m; else hi = m - 1;
  }
  return lo;
}
// The same by a whole wave, 64 probes at a time (every lane gets the result).
__device__ __forceinline__ int64_t seq_of_wave(const int32_t* __restrict__ offs, int64_t lo, int64_t hi, int64_t t) {
  const int l = lane_id();
  while (lo < hi) {
    const int64_t step = (hi - lo + WAVE - 1) / WAVE;
    const int64_t m = min(lo + step * (l + 1), hi);   // probes lo + step .. hi
    const int hits = popc(ballot(offs[m] <= t));      // offsets do not decrease: a prefix of the lanes
    const int64_t nlo = hits == 0 ? lo : min(lo + step * hits, hi);
    if (hits < WAVE) hi = min(lo + step * (hits + 1), hi) - 1;   // the first probe beyond t, less one
    lo = min(nlo, hi);
  }
  return lo;
}

// ------------------------------------------------------------------ policy loss
constexpr int POL_THREADS = 256;
constexpr int POL_TILE = 4096;      // tokens per workgroup
// One workgroup takes the whole call up to 8,192 tokens (us against the three or four launches of the general path,
// with a mask, mean over tokens / sequences: 400 tokens 8.2 / 9.1 against 12.2 / 25.9; 2,048: 9.7 / 11.9 against
// 13.3 / 17.1; 4,096: 12.1 / 15.5 against 17.6 / 22.2; 8,192: 17.0 / 22.9 against 18.5 / 22.7) ...
constexpr int POL_SMALL_N = 8192;
constexpr int POL_SMALL_SEQ = 2048; // ... and sequences (their offsets and counts lie in LDS)
constexpr int POL_SUMS = 7;         // loss, pg, kl, entropy, clipped, ratio, tokens
constexpr int POL_COUNTERS = 1024;  // workgroups that count, one partial count each (atomics on one word take
                                    // 10 ns apiece: 40 us for the waves of four million tokens)
constexpr int POL_LDS_SEQ = 1024;   // sequences of a tile whose offsets lie in LDS

struct PolArgs {
  rece_policy_config c;
  const void *logp, *old, *ref, *entropy;
  const float* adv;
  const int32_t* offs;
  const uint8_t* mask;
  const float* dloss;
  float *loss, *stats;
  void *dlogp, *dentropy;
  int32_t* part;        // [counters][2] tokens that count, sequences with such a token
  int counters;         // 0: the offsets tell (no mask, token mean)
  int32_t* cnt;         // [n_seq] tokens that count (sequence mean)
  double* partial;      // [blocks][8]
  // log(1 - clip_low), log(1 + clip_high): rounded, and what the rounding left
  float log_lo, log_lo2, log_hi, log_hi2;
};

// The values of one token.
struct PolToken {
  float lp, old, ref, H;
};
// What it adds to the sums, and its gradients by logp and entropy (without dloss).
struct PolTerm {
  float loss, pg, kl, H, r;   // loss: without the weight
  bool clipped;
  float dlp, dent;
};

// e^x to about an ulp: 2^y with y = x log2(e) rounded, times 1 + the rounding's share (y alone would leave |x| ulps).
__device__ __forceinline__ float exp_near(float x) {
  constexpr float L = 1.44269504088896341f, LLO = 1.92596299112661746e-8f;   // log2(e) and what its rounding left
  const float y = x * L;
  const float rest = fmaf(x, LLO, fmaf(x, L, -y)) * 0.693147180559945309f;
  const float e = __builtin_amdgcn_exp2f(y);
  return fabsf(y) < 200.0f ? fmaf(e, rest, e) : e;   // beyond: 0, infinity or NaN as it is
}

// em = e^u - 1 and kl = e^u - 1 - u.  Differences of e^u keep nothing of a small u, and a policy starts as its
// reference, so up to |u| = 1 the series u^2 (1/2 + u/6 + ... + u^9/11!) is summed: what it leaves out is below 2^-27
// of kl, and kl is off by at most 7 roundings (beyond |u| = 1 by 18, of which e^u has most).
__device__ __forceinline__ void kl_terms(float u, float& em, float& kl) {
  if (fabsf(u) < 1.0f) {
    float p = 1.0f / 39916800.0f;
    p = fmaf(p, u, 1.0f / 3628800.0f);
    p = fmaf(p, u, 1.0f / 362880.0f);
    p = fmaf(p, u, 1.0f / 40320.0f);
    p = fmaf(p, u, 1.0f / 5040.0f);
    p = fmaf(p, u, 1.0f / 720.0f);
    p = fmaf(p, u, 1.0f / 120.0f);
    p = fmaf(p, u, 1.0f / 24.0f);
    p = fmaf(p, u, 1.0f / 6.0f);
    p = fmaf(p, u, 0.5f);
    kl = u * u * p;
    em = u + kl;
  } else {
    em = exp_near(u) - 1.0f;
    kl = em - u;
  }
}

// One token of weight w and advantage A.
__device__ __forceinline__ PolTerm pol_token(const PolArgs& a, const PolToken& k, float w, float A) {
  PolTerm o;
  const float lo = 1.0f - a.c.clip_low, hi = 1.0f + a.c.clip_high;
  const float diff = k.lp - k.old;
  o.r = exp_near(diff);
  const float bound = A > 0.0f ? hi : lo;
  // Decided on the logarithms, with what the difference's rounding left (it is exact where the two are within a factor
  // of two, not for log-probabilities near 0) and what the bounds' left: the ratio itself is rounded, and tokens near
  // a bound would fall on the other side.  An infinite difference has no remainder.
  const float back = diff - k.lp;
  float rest = (k.lp - (diff - back)) - (k.old + back);
  rest = rest == rest ? rest : 0.0f;
  o.clipped = (A > 0.0f && diff - a.log_hi > a.log_hi2 - rest) || (A < 0.0f && diff - a.log_lo < a.log_lo2 - rest);
  o.pg = -A * (o.clipped ? bound : o.r);
  float g = o.clipped ? 0.0f : o.pg;
  o.kl = 0.0f;
  o.H = 0.0f;
  // without a coefficient a term is no part of the loss, whatever its value
  o.loss = o.pg;
  if (a.ref) {
    float em;
    kl_terms(k.ref - k.lp, em, o.kl);
    if (a.c.kl_coef != 0.0f) {
      g = fmaf(-a.c.kl_coef, em, g);
      o.loss = fmaf(a.c.kl_coef, o.kl, o.loss);
    }
  }
  if (a.entropy) {
    o.H = k.H;
    if (a.c.entropy_coef != 0.0f) o.loss = fmaf(-a.c.entropy_coef, o.H, o.loss);
  }
  o.dlp = w * g;
  o.dent = -a.c.entropy_coef * w;
  return o;
}

// Sums of a thread's tokens.
struct PolSums {
  double v[5] = {};   // loss, pg, kl, entropy, ratio
  int clipped = 0, tokens = 0;
  __device__ __forceinline__ void add(const PolTerm& o, bool on, double w) {
    v[0] = fma((double)(on ? o.loss : 0.0f), w, v[0]);
    v[1] += on ? o.pg : 0.0f;
    v[2] += on ? o.kl : 0.0f;
    v[3] += on ? o.H : 0.0f;
    v[4] += on ? o.r : 0.0f;
    clipped += on && o.clipped ? 1 : 0;
    tokens += on ? 1 : 0;
  }
  __device__ __forceinline__ void get(double (&o)[POL_SUMS]) const {
    o[0] = v[0], o[1] = v[1], o[2] = v[2], o[3] = v[3], o[4] = clipped, o[5] = v[4], o[6] = tokens;
  }
};

__global__ __launch_bounds__(POL_THREADS) void k_pol_clear(int32_t* __restrict__ p, int64_t n) {
  const int64_t t = (int64_t)blockIdx.x * POL_THREADS + threadIdx.x;
  if (t < n) p[t] = 0;
}

// Tokens that count: all (token mean) or per sequence, and the sequences that have one.
__global__ __launch_bounds__(POL_THREADS) void k_pol_count(PolArgs a) {
  constexpr int PER = POL_TILE / POL_THREADS;
  __shared__ int sh[2][POL_THREADS / WAVE];
  const int64_t n = a.c.n, ns = a.c.n_seq;
  const int64_t first = offset_at(a.offs, 0, n), end = offset_at(a.offs, ns, n);
  const bool per_seq = a.c.reduction == RECE_MEAN_SEQUENCE;
  int tokens = 0, with = 0;
  auto add = [&](int64_t s, int c) { with += atomicAdd(&a.cnt[s], c) == 0 ? 1 : 0; };   // whoever finds 0 counts the sequence
  for (int64_t base = (int64_t)blockIdx.x * POL_TILE; base < n; base += (int64_t)gridDim.x * POL_TILE) {
    const int64_t t0 = base + (int64_t)threadIdx.x * PER;
    const int64_t lo = max(first, t0), hi = min(end, min(n, t0 + PER));
    uint32_t bits = 0;
    if (lo < hi) {
      if (!a.mask) {
        bits = ((1u << (hi - t0)) - 1u) & ~((1u << (lo - t0)) - 1u);
      } else if (hi - t0 == PER && (reinterpret_cast<uintptr_t>(a.mask) & 15) == 0) {
        const u32x4 m = *reinterpret_cast<const u32x4*>(a.mask + t0);
#pragma unroll
        for (int q = 0; q < PER; ++q) bits |= ((m[q / 4] >> (8 * (q % 4))) & 0xFFu) ? 1u << q : 0u;
        bits &= ~((1u << (lo - t0)) - 1u);
      } else {
        for (int64_t t = lo; t < hi; ++t) bits |= a.mask[t] ? 1u << (t - t0) : 0u;
      }
    }
    tokens += __popc(bits);
    if (!per_seq) continue;
    const int64_t wave0 = base + (int64_t)(threadIdx.x & ~(WAVE - 1)) * PER;
    if (wave0 >= n) continue;   // whole waves
    const int64_t s0 = seq_of_wave(a.offs, 0, ns - 1, wave0);
    const int64_t s1 = seq_of_wave(a.offs, s0, ns - 1, min(n, wave0 + WAVE * PER) - 1);
    if (s1 - s0 < 16) {   // few sequences: one atomic each per wave (64 lanes on one word cost 30 us more for 4.2M tokens)
      for (int64_t s = s0; s <= s1; ++s) {
        const int64_t b = s == s0 ? t0 : max(t0, offset_at(a.offs, s, n)), e = s == s1 ? t0 + PER : offset_at(a.offs, s + 1, n);
        const int64_t from = min(b - t0, (int64_t)PER), to = min(max(e - t0, (int64_t)0), (int64_t)PER);
        const int c = wave_sum(from < to ? __popc(bits & ((1u << to) - 1u) & ~((1u << from) - 1u)) : 0);
        if (lane_id() == 0 && c) add(s, c);
      }
      continue;
    }
    int64_t t = lo;
    while (t < hi) {
      const int64_t s = seq_of(a.offs, s0, s1, t);
      const int64_t e = max(t + 1, min(hi, offset_at(a.offs, s + 1, n)));
      const uint32_t part = bits & ~((1u << (t - t0)) - 1u) & (e - t0 >= 32 ? ~0u : (1u << (e - t0)) - 1u);
      if (part) add(s, __popc(part));
      t = e;
    }
  }
  tokens = wave_sum(tokens);
  with = wave_sum(with);
  if (lane_id() == 0) {
    sh[0][threadIdx.x / WAVE] = tokens;
    sh[1][threadIdx.x / WAVE] = with;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < POL_THREADS / WAVE; ++w) c += sh[threadIdx.x][w];
    a.part[blockIdx.x * 2 + threadIdx.x] = c;
  }
}

__device__ __forceinline__ void pol_write(const PolArgs& a, const double (&v)[POL_SUMS]) {
  const double m = v[6] > 0.0 ? 1.0 / v[6] : 0.0;
  a.loss[0] = (float)v[0];
#pragma unroll
  for (int k = 1; k < 6; ++k) a.stats[k - 1] = (float)(v[k] * m);
  a.stats[5] = (float)v[6];
}

// Sums of v over the workgroup in a fixed order, in thread 0.
template <int NT>
__device__ __forceinline__ void pol_reduce(double (&v)[POL_SUMS], double (*sh)[POL_SUMS]) {
#pragma unroll
  for (int k = 0; k < POL_SUMS; ++k) v[k] = wave_sum_d(v[k]);
  __syncthreads();
  if (lane_id() == 0)
#pragma unroll
    for (int k = 0; k < POL_SUMS; ++k) sh[threadIdx.x / WAVE][k] = v[k];
  __syncthreads();
  if (threadIdx.x == 0)
#pragma unroll
    for (int k = 0; k < POL_SUMS; ++k) {
      v[k] = 0.0;
      for (int w = 0; w < NT / WAVE; ++w) v[k] += sh[w][k];
    }
}

// W consecutive values of a token array, W = 4 with one load or store (the array and t aligned to it).
template <int W>
__device__ __forceinline__ void load_tokens(const float* p, int64_t t, float (&v)[W]) {
  if constexpr (W == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p + t);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
    v[0] = p[t];
  }
}
template <int W>
__device__ __forceinline__ void load_tokens(const bf16* p, int64_t t, float (&v)[W]) {
  if constexpr (W == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p + t);
    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xFFFF0000u);
    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xFFFF0000u);
  } else {
    v[0] = to_f32(p[t]);
  }
}
// 0x80 in byte e: token t + e counts.
template <int W>
__device__ __forceinline__ uint32_t load_mask(const uint8_t* p, int64_t t) {
  if constexpr (W == 4) {
    if (!p) return 0x80808080u;
    const uint32_t m = *reinterpret_cast<const uint32_t*>(p + t);
    return (((m & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | m) & 0x80808080u;
  } else {
    return !p || p[t] ? 0x80u : 0u;
  }
}
template <int W>
__device__ __forceinline__ void store_tokens(float* p, int64_t t, const float (&v)[W]) {
  if constexpr (W == 4)
    *reinterpret_cast<float4*>(p + t) = float4{v[0], v[1], v[2], v[3]};
  else
    p[t] = v[0];
}
template <int W>
__device__ __forceinline__ void store_tokens(bf16* p, int64_t t, const float (&v)[W]) {
  if constexpr (W == 4)
    *reinterpret_cast<uint2*>(p + t) = uint2{bf16_of(v[0]) | (bf16_of(v[1]) << 16), bf16_of(v[2]) | (bf16_of(v[3]) << 16)};
  else
    p[t].bits = (uint16_t)bf16_of(v[0]);
}

// A tile of tokens per workgroup, W consecutive ones per thread and step; the tile's values are requested before
// anything waits for counts or offsets, and what a token needs of its sequence lies in LDS.
template <class E, int W>
__global__ __launch_bounds__(POL_THREADS) void k_pol_main(PolArgs a) {
  constexpr int STEPS = POL_TILE / POL_THREADS / W;
  constexpr int GROUP = 4;   // steps whose values are in flight together
  static_assert(STEPS % GROUP == 0, "tile");
  __shared__ double sh[POL_THREADS / WAVE][POL_SUMS];
  __shared__ int32_t soff[POL_LDS_SEQ + 1];
  __shared__ float sadv[POL_LDS_SEQ];
  __shared__ double sw[POL_LDS_SEQ];
  __shared__ int64_t srange[2];
  __shared__ int scount[2][POL_THREADS / WAVE];
  const uint32_t n = (uint32_t)a.c.n, ns = (uint32_t)a.c.n_seq;   // below 2^31: a tile beyond fits in 32 bits
  const uint32_t lo = (uint32_t)offset_at(a.offs, 0, n), hi = (uint32_t)offset_at(a.offs, ns, n);
  const uint32_t base = blockIdx.x * POL_TILE;
  const int tid = threadIdx.x, wave = tid / WAVE;
  const bool per_seq = a.c.reduction == RECE_MEAN_SEQUENCE, seq_adv = !a.c.token_adv, need_seq = per_seq || seq_adv;
  float lp[GROUP][W], old[GROUP][W], ref[GROUP][W], ent[GROUP][W];
  uint32_t on[GROUP];
  const bool inside = lo <= base && base + POL_TILE <= hi;   // every token of the tile lies in a sequence
  auto load = [&](int g) {
#pragma unroll
    for (int u = 0; u < GROUP; ++u) {
      const uint32_t t = base + ((g + u) * POL_THREADS + tid) * W;
      on[u] = 0;
#pragma unroll
      for (int e = 0; e < W; ++e) lp[u][e] = old[u][e] = ref[u][e] = ent[u][e] = 0.0f;
      if (t + W <= n) {
        load_tokens<W>(static_cast<const E*>(a.logp), t, lp[u]);
        load_tokens<W>(static_cast<const E*>(a.old), t, old[u]);
        if (a.ref) load_tokens<W>(static_cast<const E*>(a.ref), t, ref[u]);
        if (a.entropy) load_tokens<W>(static_cast<const E*>(a.entropy), t, ent[u]);
        on[u] = load_mask<W>(a.mask, t);
      } else if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (t + e < n) {
            lp[u][e] = to_f32(static_cast<const E*>(a.logp)[t + e]);
            old[u][e] = to_f32(static_cast<const E*>(a.old)[t + e]);
            if (a.ref) ref[u][e] = to_f32(static_cast<const E*>(a.ref)[t + e]);
            if (a.entropy) ent[u][e] = to_f32(static_cast<const E*>(a.entropy)[t + e]);
            on[u] |= load_mask<1>(a.mask, t + e) << (8 * e);
          }
      }
      if (!inside)
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (t + e < lo || t + e >= hi) on[u] &= ~(0x80u << (8 * e));
    }
  };
  load(0);
  const float up = a.dloss ? a.dloss[0] : 1.0f;
  if (a.counters) {
    int c0 = 0, c1 = 0;
    for (int q = tid; q < a.counters; q += POL_THREADS) {
      const int2 c = reinterpret_cast<const int2*>(a.part)[q];
      c0 += c.x;
      c1 += c.y;
    }
    c0 = wave_sum(c0);
    c1 = wave_sum(c1);
    if (lane_id() == 0) {
      scount[0][wave] = c0;
      scount[1][wave] = c1;
    }
  }
  if (need_seq && wave < 2) {   // the sequences of the tile's first and last token
    const int64_t s = seq_of_wave(a.offs, 0, (int64_t)ns - 1, wave == 0 ? base : min(n, base + POL_TILE) - 1);
    if (lane_id() == 0) srange[wave] = s;
  }
  __syncthreads();
  int tokens = hi > lo ? (int)(hi - lo) : 0, with = 0;
  if (a.counters) {
    tokens = 0;
#pragma unroll
    for (int w = 0; w < POL_THREADS / WAVE; ++w) {
      tokens += scount[0][w];
      with += scount[1][w];
    }
  }
  const double wt = 1.0 / (double)max(tokens, 1), nonempty = (double)max(with, 1);
  const uint32_t s0 = need_seq ? (uint32_t)srange[0] : 0, s1 = need_seq ? max(s0, (uint32_t)srange[1]) : 0;
  const bool in_lds = s1 - s0 < POL_LDS_SEQ;
  auto weight_of = [&](uint32_t sq) { return per_seq ? 1.0 / ((double)max(a.cnt[sq], 1) * nonempty) : wt; };
  if (need_seq && in_lds)
    for (uint32_t q = tid; q <= s1 - s0 + 1; q += POL_THREADS) {
      soff[q] = a.offs[s0 + q];
      if (q <= s1 - s0) {
        sadv[q] = seq_adv ? a.adv[s0 + q] : 0.0f;
        sw[q] = weight_of(s0 + q);
      }
    }
  __syncthreads();
  PolSums s;
#pragma unroll 1
  for (int g = 0; g < STEPS; g += GROUP) {
    if (g > 0) load(g);
#pragma unroll
    for (int u = 0; u < GROUP; ++u) {
      const uint32_t t = base + ((g + u) * POL_THREADS + tid) * W;
      if (t >= n) continue;
      float dlp[W], dent[W], A[W];
      double w[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        A[e] = 0.0f;
        w[e] = wt;
      }
      if (need_seq) {
        int64_t until = 0;   // the end of the sequence before
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (e > 0) {
            A[e] = A[e - 1];
            w[e] = w[e - 1];
          }
          const uint32_t te = t + e;
          if (e > 0 && (int64_t)te < until) continue;
          if (in_lds) {
            int l = 0, h = (int)(s1 - s0);
            while (l < h) {
              const int m = (l + h + 1) / 2;
              if (soff[m] <= (int)te) l = m; else h = m - 1;
            }
            until = soff[l + 1];
            A[e] = sadv[l];
            w[e] = sw[l];
          } else {
            const int64_t sq = seq_of(a.offs, s0, s1, te);
            until = a.offs[sq + 1];
            if (seq_adv) A[e] = a.adv[sq];
            w[e] = weight_of((uint32_t)sq);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const bool live = (on[u] >> (8 * e)) & 0x80u;
        if (!seq_adv) A[e] = live ? a.adv[t + e] : 0.0f;
        const PolTerm o = pol_token(a, PolToken{lp[u][e], old[u][e], ref[u][e], ent[u][e]}, (float)w[e], A[e]);
        s.add(o, live, w[e]);   // what lies at a token that does not count is selected away, NaN included
        dlp[e] = live ? up * o.dlp : 0.0f;
        dent[e] = live ? up * o.dent : 0.0f;
      }
      if (t + W <= n) {
        if (a.dlogp) store_tokens<W>(static_cast<E*>(a.dlogp), t, dlp);
        if (a.dentropy) store_tokens<W>(static_cast<E*>(a.dentropy), t, dent);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (t + e < n) {
            if (a.dlogp) put(static_cast<E*>(a.dlogp), t + e, dlp[e]);
            if (a.dentropy) put(static_cast<E*>(a.dentropy), t + e, dent[e]);
          }
      }
    }
  }
  double v[POL_SUMS];
  s.get(v);
  pol_reduce<POL_THREADS>(v, sh);
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < POL_SUMS; ++k) a.partial[(int64_t)blockIdx.x * 8 + k] = v[k];
  }
}

// The workgroups' sums, in their order.
__global__ __launch_bounds__(POL_THREADS) void k_pol_final(PolArgs a, int64_t blocks) {
  __shared__ double sh[POL_THREADS / WAVE][POL_SUMS];
  double v[POL_SUMS];
#pragma unroll
  for (int k = 0; k < POL_SUMS; ++k) v[k] = 0.0;
#pragma unroll 4
  for (int64_t b = threadIdx.x; b < blocks; b += POL_THREADS)
#pragma unroll
    for (int k = 0; k < POL_SUMS; ++k) v[k] += a.partial[b * 8 + k];
  pol_reduce<POL_THREADS>(v, sh);
  if (threadIdx.x == 0) pol_write(a, v);
}

// The whole call in one workgroup: counts in LDS, then the tokens.
constexpr int POL_SMALL_THREADS = 1024;
template <class E>
__global__ __launch_bounds__(POL_SMALL_THREADS) void k_pol_small(PolArgs a) {
  constexpr int PER = POL_SMALL_N / POL_SMALL_THREADS;
  __shared__ int32_t offs[POL_SMALL_SEQ + 1];
  __shared__ int32_t cnt[POL_SMALL_SEQ];
  __shared__ double sh[POL_SMALL_THREADS / WAVE];
  __shared__ double sums[POL_SMALL_THREADS / WAVE][POL_SUMS];
  const int n = (int)a.c.n, ns = (int)a.c.n_seq;
  const bool per_seq = a.c.reduction == RECE_MEAN_SEQUENCE;
  for (int i = threadIdx.x; i <= ns; i += POL_SMALL_THREADS) {
    offs[i] = (int32_t)offset_at(a.offs, i, n);
    if (i < ns) cnt[i] = 0;
  }
  // every value is requested before the first is used
  PolToken k[PER];
  bool in[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int t = q * POL_SMALL_THREADS + (int)threadIdx.x;
    in[q] = t < n && (!a.mask || a.mask[t < n ? t : 0]);
    k[q] = PolToken{};
    if (t < n) {
      k[q].lp = to_f32(static_cast<const E*>(a.logp)[t]);
      k[q].old = to_f32(static_cast<const E*>(a.old)[t]);
      if (a.ref) k[q].ref = to_f32(static_cast<const E*>(a.ref)[t]);
      if (a.entropy) k[q].H = to_f32(static_cast<const E*>(a.entropy)[t]);
    }
  }
  __syncthreads();
  int sq[PER];
  float A[PER];
  int mine = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int t = q * POL_SMALL_THREADS + (int)threadIdx.x;
    sq[q] = -1;
    A[q] = 0.0f;
    if (in[q] && t >= offs[0] && t < offs[ns]) {
      int lo = 0, hi = ns - 1;
      while (lo < hi) {
        const int m = (lo + hi + 1) / 2;
        if (offs[m] <= t) lo = m; else hi = m - 1;
      }
      sq[q] = lo;
      A[q] = a.adv[a.c.token_adv ? t : lo];
      ++mine;
      if (per_seq) atomicAdd(&cnt[lo], 1);
    }
  }
  const double tokens = block_sum_d<POL_SMALL_THREADS>((double)mine, sh);   // also: the counts are complete
  double with = 0.0;
  if (per_seq) {
    for (int i = threadIdx.x; i < ns; i += POL_SMALL_THREADS) with += cnt[i] > 0 ? 1.0 : 0.0;
    with = block_sum_d<POL_SMALL_THREADS>(with, sh);
  }
  const double wt = 1.0 / fmax(tokens, 1.0), nonempty = fmax(with, 1.0);
  const float up = a.dloss ? a.dloss[0] : 1.0f;
  PolSums s;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int t = q * POL_SMALL_THREADS + (int)threadIdx.x;
    if (t >= n) break;
    float dlp = 0.0f, dent = 0.0f;
    if (sq[q] >= 0) {
      const double w = per_seq ? 1.0 / ((double)cnt[sq[q]] * nonempty) : wt;
      const PolTerm o = pol_token(a, k[q], (float)w, A[q]);
      s.add(o, true, w);
      dlp = o.dlp;
      dent = o.dent;
    }
    const bool live = sq[q] >= 0;   // others get 0 whatever dloss is
    if (a.dlogp) put(static_cast<E*>(a.dlogp), t, live ? up * dlp : 0.0f);
    if (a.dentropy) put(static_cast<E*>(a.dentropy), t, live ? up * dent : 0.0f);
  }
  double v[POL_SUMS];
  s.get(v);
  pol_reduce<POL_SMALL_THREADS>(v, sums);
  if (threadIdx.x == 0) pol_write(a, v);
}

// ------------------------------------------------------------------ preference loss
struct PrefArgs {
  rece_preference_config c;
  const void *logp, *ref;
  const int32_t *offs, *goffs;
  const uint8_t* mask;
  const float* dloss;
  double* group_loss;   // [n_group]
  double* h;            // [n_seq]
  double* share;        // [n_seq] 1, or 1 / tokens that count (average)
  float *loss, *loss_pg, *rewards;
  void* dlogp;
};

// Tokens [lo, hi) of a sequence; tokens are below 2^31, so a step beyond fits in 32 bits.
struct PrefSeq {
  uint32_t lo, hi;
};
__device__ __forceinline__ PrefSeq pref_seq(const int32_t* offs, int64_t i, int64_t n) {
  const uint32_t lo = (uint32_t)offset_at(offs, i, n), hi = (uint32_t)offset_at(offs, i + 1, n);
  return PrefSeq{lo, max(lo, hi)};
}

// 0x80 in byte e: token t + e lies in the sequence (t in [lo / W * W, hi)).
template <int W>
__device__ __forceinline__ uint32_t pref_in(PrefSeq q, uint32_t t) {
  if constexpr (W == 1) return 0x80u;
  uint32_t in = 0x80808080u;
  if (t < q.lo) in &= ~0u << (8 * (q.lo - t));
  if (q.hi - t < 4) in &= ~0u >> (8 * (4 - (q.hi - t)));
  return in;
}

// A few lanes take PREF_STEPS steps of their sequence by themselves; what is left of a longer one the whole wave takes
// (lengths are known on the device alone, and a mean of two says nothing of the longest: one sequence of 10,000 tokens
// among 100,000 of two 1,680 us by its own lane, 53 by the wave).
constexpr int PREF_STEPS = 32;

// First token of the part that the wave takes; hi where there is none.
template <int L, int W>
__device__ __forceinline__ uint32_t pref_rest(PrefSeq q) {
  if constexpr (L == WAVE) return q.hi;
  return min((uint64_t)q.hi, (uint64_t)(q.lo / W * W) + (uint64_t)PREF_STEPS * L * W);
}

// f(lane, first token, end) for the lane that speaks for each sequence with such a part, by the whole wave.
template <int L, class F>
__device__ __forceinline__ void pref_rests(uint32_t from, uint32_t hi, int sub, F f) {
  for (uint64_t left = ballot(sub == 0 && from < hi); left; left &= left - 1) {
    const int lane = __ffsll((unsigned long long)left) - 1;
    f(lane, __builtin_amdgcn_readlane(from, lane), __builtin_amdgcn_readlane(hi, lane));
  }
}

// h of K sequences by L lanes (all of them get them); the K sequences' tokens are requested together.  All lanes of a
// wave come here together, those without a sequence with an empty one.
template <class E, int L, int W, int K>
__device__ __forceinline__ void pref_sum(const PrefArgs& a, const PrefSeq (&whole)[K], int sub, double (&s)[K], double (&share)[K]) {
  const E* lp = static_cast<const E*>(a.logp);
  const E* rf = static_cast<const E*>(a.ref);
  const uint32_t n = (uint32_t)a.c.n;
  int c[K];
  uint32_t t[K];
  PrefSeq seq[K];   // the part that the lanes take by themselves
  bool more = false;
#pragma unroll
  for (int q = 0; q < K; ++q) {
    seq[q] = PrefSeq{whole[q].lo, pref_rest<L, W>(whole[q])};
    s[q] = 0.0;
    c[q] = 0;
    t[q] = seq[q].lo / W * W + sub * W;
    more |= t[q] < seq[q].hi;
  }
  while (more) {
    float x[K][W], y[K][W];
    uint32_t on[K];
#pragma unroll
    for (int q = 0; q < K; ++q) {
#pragma unroll
      for (int e = 0; e < W; ++e) x[q][e] = y[q][e] = 0.0f;
      on[q] = 0;
      if (t[q] >= seq[q].hi) continue;
      if (t[q] + W <= n) {
        load_tokens<W>(lp, t[q], x[q]);
        if (rf) load_tokens<W>(rf, t[q], y[q]);
        on[q] = load_mask<W>(a.mask, t[q]);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (t[q] + e < n) {
            x[q][e] = to_f32(lp[t[q] + e]);
            if (rf) y[q][e] = to_f32(rf[t[q] + e]);
            on[q] |= load_mask<1>(a.mask, t[q] + e) << (8 * e);
          }
      }
    }
    more = false;
#pragma unroll
    for (int q = 0; q < K; ++q) {
      if (t[q] >= seq[q].hi) continue;
      on[q] &= pref_in<W>(seq[q], t[q]);
#pragma unroll
      for (int e = 0; e < W; ++e) s[q] += (double)((on[q] >> (8 * e)) & 0x80u ? x[q][e] - y[q][e] : 0.0f);
      c[q] += __popc(on[q]);
      t[q] += L * W;
      more |= t[q] < seq[q].hi;
    }
  }
  if constexpr (L < WAVE) {
#pragma unroll
    for (int q = 0; q < K; ++q)
      pref_rests<L>(seq[q].hi, whole[q].hi, sub, [&](int lane, uint32_t from, uint32_t hi) {
        constexpr int UNR = 8;   // tokens of a lane in flight
        double v = 0.0;
        int on = 0;
        for (uint32_t t0 = from; t0 < hi; t0 += UNR * WAVE) {
          float x[UNR], y[UNR];
          bool in[UNR];
#pragma unroll
          for (int u = 0; u < UNR; ++u) {
            const uint32_t at = t0 + u * WAVE + lane_id();
            in[u] = at < hi && (!a.mask || a.mask[at]);
            x[u] = at < hi ? to_f32(lp[at]) : 0.0f;
            y[u] = at < hi && rf ? to_f32(rf[at]) : 0.0f;
          }
#pragma unroll
          for (int u = 0; u < UNR; ++u) {
            v += (double)(in[u] ? x[u] - y[u] : 0.0f);
            on += in[u] ? 1 : 0;
          }
        }
        v = wave_sum_d(v);
        on = wave_sum(on);
        if (lane_id() == lane) {
          s[q] += v;
          c[q] += on;
        }
      });
  }
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1)
#pragma unroll
    for (int q = 0; q < K; ++q) s[q] += __shfl_xor(s[q], o);
#pragma unroll
  for (int q = 0; q < K; ++q) {
    share[q] = 1.0;
    if (a.c.average) {
#pragma unroll
      for (int o = L / 2; o >= 1; o >>= 1) c[q] += __shfl_xor(c[q], o);
      share[q] = 1.0 / (double)max(c[q], 1);
      s[q] /= (double)max(c[q], 1);
    }
  }
}

// Gradient of a sequence's tokens: v where they count, else 0.  All lanes of a wave come here together.
template <class E, int L, int W>
__device__ __forceinline__ void pref_grad(const PrefArgs& a, PrefSeq whole, int sub, float v) {
  E* out = static_cast<E*>(a.dlogp);
  const PrefSeq seq{whole.lo, pref_rest<L, W>(whole)};
  if constexpr (L < WAVE)
    pref_rests<L>(seq.hi, whole.hi, sub, [&](int lane, uint32_t from, uint32_t hi) {
      const float x = __shfl(v, lane);
      for (uint32_t t = from + lane_id(); t < hi; t += WAVE) put(out, t, load_mask<1>(a.mask, t) ? x : 0.0f);
    });
  for (uint32_t t = seq.lo / W * W + sub * W; t < seq.hi; t += L * W) {
    const uint32_t in = pref_in<W>(seq, t);
    if (W == 1 || in == 0x80808080u) {   // inside the sequence, so inside the array
      const uint32_t on = load_mask<W>(a.mask, t);
      float x[W];
#pragma unroll
      for (int e = 0; e < W; ++e) x[e] = (on >> (8 * e)) & 0x80u ? v : 0.0f;
      store_tokens<W>(out, t, x);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e)
        if ((in >> (8 * e)) & 0x80u) put(out, t + e, load_mask<1>(a.mask, t + e) ? v : 0.0f);
    }
  }
}

// log(1 + sum of e^v) from top, the largest v or 0, and the sum of e^(v - top): small where every v is far below 0.
__device__ __forceinline__ double softmax_loss(double top, double others) {
  return top > 0.0 ? top + log(others + exp(-top)) : log1p(others);
}

// e^(v - top) with top the largest: 1 for v = top, also where both are infinite.
__device__ __forceinline__ double exp_below(double v, double top) { return exp(v == top ? 0.0 : v - top); }

__device__ __forceinline__ double softplus_d(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

// Loss of one pair and its derivative by z.
__device__ __forceinline__ double pair_loss(const rece_preference_config& c, double z, double& dz) {
  if (c.kind == RECE_PREF_SIGMOID) {
    const double e = c.smoothing;
    dz = e - 1.0 / (1.0 + exp(z));   // as sigmoid(z) - (1 - e) nothing would be left of it where z is large
    // without smoothing its term is no part of the loss, also where z is infinite (an item of no probability)
    return (1.0 - e) * softplus_d(-z) + (e > 0.0 ? e * softplus_d(z) : 0.0);
  }
  if (c.kind == RECE_PREF_IPO) {
    const double b = c.beta, v = z / b - 0.5 / b;
    dz = 2.0 * v / b;
    return v * v;
  }
  // comparisons that leave a NaN a NaN
  const double v = 1.0 - z;
  dz = v > 0.0 ? -1.0 : v <= 0.0 ? 0.0 : v;
  return v < 0.0 ? 0.0 : v;
}

constexpr int PREF_LDS = 512;   // sequences of a group whose h lies in LDS
constexpr int64_t PREF_MANY = 8192, PREF_PAIRS = 2048;   // groups (pairs) above which small ones share waves
constexpr int PREF_EXTRA = 1024; // workgroups for what lies in no group

// What lies in no group, by workgroup b of `extra`: the rewards of its sequences, gradients of zero.
template <class E, int L, int W, int NT>
__device__ __forceinline__ void pref_outside(const PrefArgs& a, int64_t b, int64_t extra) {
  constexpr int NS = NT / L;   // sequences at a time
  const int64_t G = a.c.n_group, nseq = a.c.n_seq;
  const int q = threadIdx.x / L, sub = threadIdx.x % L;
  const float beta = a.c.beta;
  const int64_t first = offset_at(a.goffs, 0, nseq), end = offset_at(a.goffs, G, nseq);
  for (int64_t k0 = b * NS; k0 < first + (nseq - end); k0 += extra * NS) {   // lanes together
    const int64_t k = k0 + q, i = k < first ? k : end + (k - first);
    const bool on = k < first + (nseq - end) && i < nseq;
    const PrefSeq seq[1] = {on ? pref_seq(a.offs, i, a.c.n) : PrefSeq{0, 0}};
    double h[1], share[1];
    pref_sum<E, L, W, 1>(a, seq, sub, h, share);
    if (on && sub == 0) a.rewards[i] = (float)((double)beta * h[0]);
    if (a.dlogp) pref_grad<E, L, W>(a, seq[0], sub, 0.0f);
  }
  if (a.dlogp) {
    const int64_t lo = offset_at(a.offs, 0, a.c.n), hi = max(lo, offset_at(a.offs, nseq, a.c.n));
    for (int64_t k = b * NT + threadIdx.x; k < lo + (a.c.n - hi); k += extra * NT)
      put(static_cast<E*>(a.dlogp), k < lo ? k : hi + (k - lo), 0.0f);
  }
}

// The last n_group workgroups: one group each.  Those before: the sequences in no group, and the tokens in no
// sequence.
template <class E, int L, int W, int NT>
__global__ __launch_bounds__(NT) void k_pref(PrefArgs a, int extra) {
  constexpr int NS = NT / L;   // sequences at a time
  __shared__ double sh_h[PREF_LDS];
  __shared__ double sh_share[PREF_LDS];
  __shared__ int32_t sh_offs[PREF_LDS + 1];
  const int64_t G = a.c.n_group, nseq = a.c.n_seq;
  const int q = threadIdx.x / L, sub = threadIdx.x % L;
  const float beta = a.c.beta;
  const int64_t blk = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (blk >= extra + G) return;
  if (blk < extra) {
    pref_outside<E, L, W, NT>(a, blk, extra);
    return;
  }
  const int64_t g = blk - extra;
  const int64_t s0 = offset_at(a.goffs, g, nseq), s1 = max(s0, offset_at(a.goffs, g + 1, nseq));
  const int64_t m = s1 - s0;
  const bool in_lds = m <= PREF_LDS;
  if (in_lds) {
    for (int64_t k = threadIdx.x; k <= m; k += NT) sh_offs[k] = a.offs[s0 + k];
    __syncthreads();
  }
  auto seq_at = [&](int64_t k) { return in_lds ? pref_seq(sh_offs, k, a.c.n) : pref_seq(a.offs, s0 + k, a.c.n); };
  for (int64_t k0 = 0; k0 < m; k0 += 2 * NS) {   // lanes together
    const int64_t k = k0 + q;
    const PrefSeq seq[2] = {k < m ? seq_at(k) : PrefSeq{0, 0}, k + NS < m ? seq_at(k + NS) : PrefSeq{0, 0}};
    double h[2], share[2];
    pref_sum<E, L, W, 2>(a, seq, sub, h, share);
    if (sub != 0) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t i = k + u * NS;
      if (i >= m) break;
      a.rewards[s0 + i] = (float)((double)beta * h[u]);
      if (in_lds) {
        sh_h[i] = h[u];
        sh_share[i] = share[u];
      } else {
        a.h[s0 + i] = h[u];
        a.share[s0 + i] = share[u];
      }
    }
  }
  __syncthreads();
  // The first wave takes the group's loss, a member per lane, and leaves the derivatives by h where the h were.
  double* hs = in_lds ? sh_h : a.h + s0;
  const double* shares = in_lds ? sh_share : a.share + s0;
  if (threadIdx.x < WAVE) {
    const int l = lane_id();
    double loss = 0.0, dc = 0.0;
    if (m >= 2) {
      const double hc = hs[0], per = 1.0 / (double)(m - 1);
      auto z_of = [&](int64_t k) { return (double)beta * (hc - hs[k]) - (double)a.c.margin; };
      if (a.c.kind == RECE_PREF_SOFTMAX) {
        double top = 0.0, others = 0.0;
        for (int64_t k = 1 + l; k < m; k += WAVE) top = fmax(top, -z_of(k));
        top = wave_max_d(top);
        for (int64_t k = 1 + l; k < m; k += WAVE) {
          const double e = exp_below(-z_of(k), top);
          others += e;
          hs[k] = e;
        }
        others = wave_sum_d(others);
        const double tot = others + exp(-top);
        for (int64_t k = 1 + l; k < m; k += WAVE) hs[k] = hs[k] / tot;
        loss = softmax_loss(top, others);
        dc = -others / tot;
      } else {
        for (int64_t k = 1 + l; k < m; k += WAVE) {
          double dz;
          loss += pair_loss(a.c, z_of(k), dz);
          dc += dz;
          hs[k] = -dz * per;
        }
        loss = wave_sum_d(loss) * per;
        dc = wave_sum_d(dc) * per;
      }
    }
    if (l == 0) {
      a.loss_pg[g] = (float)loss;
      a.group_loss[g] = loss;
      if (m > 0) hs[0] = dc;
    }
  }
  if (!a.dlogp) return;
  __syncthreads();
  const double up = (double)beta * (a.dloss ? (double)a.dloss[0] : 1.0) / (double)G;
  for (int64_t k0 = 0; k0 < m; k0 += NS) {
    const int64_t k = k0 + q;
    const bool on = k < m;
    pref_grad<E, L, W>(a, on ? seq_at(k) : PrefSeq{0, 0}, sub, on ? (float)(hs[k] * up * shares[k]) : 0.0f);
  }
}

// Many small groups: T lanes take a group, its sequences one after the other.
constexpr int PREF_MANY_THREADS = 256;
template <class E, int T, int W>
__global__ __launch_bounds__(PREF_MANY_THREADS) void k_pref_many(PrefArgs a, int extra) {
  const int64_t blk = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (blk < extra) {
    pref_outside<E, T, W, PREF_MANY_THREADS>(a, blk, extra);
    return;
  }
  const int64_t G = a.c.n_group, nseq = a.c.n_seq;
  const int64_t g = (blk - extra) * (PREF_MANY_THREADS / T) + threadIdx.x / T;
  const int sub = threadIdx.x % T;
  const bool there = g < G;
  const int64_t s0 = there ? offset_at(a.goffs, g, nseq) : 0, s1 = there ? max(s0, offset_at(a.goffs, g + 1, nseq)) : 0;
  const int64_t m = s1 - s0;
  const double beta = a.c.beta, margin = a.c.margin;
  const double up = beta * (a.dloss ? (double)a.dloss[0] : 1.0) / (double)G, per = m > 1 ? 1.0 / (double)(m - 1) : 0.0;
  PrefSeq seq[1];
  double h[1], share[1];
  auto read = [&](int64_t k) {   // lanes together, also those whose group has fewer members
    seq[0] = k < m ? pref_seq(a.offs, s0 + k, a.c.n) : PrefSeq{0, 0};
    pref_sum<E, T, W, 1>(a, seq, sub, h, share);
    if (k < m && sub == 0) a.rewards[s0 + k] = (float)(beta * h[0]);
  };
  const int64_t most = wave_max_i((int)m);   // the wave's largest group
  auto grad = [&](double dh) {   // of the sequence read last
    if (a.dlogp) pref_grad<E, T, W>(a, seq[0], sub, (float)(dh * up * share[0]));
  };
  double loss = 0.0, dc = 0.0;
  read(0);
  const double hc = h[0], share0 = share[0];
  const PrefSeq seq0 = seq[0];
  if (a.c.kind == RECE_PREF_SOFTMAX) {
    double top = 0.0, others = 0.0;   // others: sum of e^(-z - top)
    for (int64_t k = 1; k < most; ++k) {
      read(k);
      if (k >= m) continue;
      const double v = margin - beta * (hc - h[0]);
      if (v > top) {
        others *= exp(top - v);
        top = v;
      }
      others += exp_below(v, top);
    }
    const double tot = others + exp(-top);
    if (m > 1) {
      loss = softmax_loss(top, others);
      dc = -others / tot;
    }
    if (a.dlogp)
      for (int64_t k = 1; k < most; ++k) {
        read(k);
        grad(exp_below(margin - beta * (hc - h[0]), top) / tot);
      }
  } else {
    for (int64_t k = 1; k < most; ++k) {
      read(k);
      double dz = 0.0;
      if (k < m) {
        loss += pair_loss(a.c, beta * (hc - h[0]) - margin, dz);
        dc += dz;
      }
      grad(-dz * per);
    }
    loss *= per;
    dc *= per;
  }
  seq[0] = seq0;
  share[0] = share0;
  grad(dc);
  if (there && sub == 0) {
    a.loss_pg[g] = (float)loss;
    a.group_loss[g] = loss;
  }
}

constexpr int PREF_MEAN_THREADS = 1024;
__global__ __launch_bounds__(PREF_MEAN_THREADS) void k_pref_mean(PrefArgs a) {
  __shared__ double sh[PREF_MEAN_THREADS / WAVE];
  double v = 0.0;
#pragma unroll 4
  for (int64_t g = threadIdx.x; g < a.c.n_group; g += PREF_MEAN_THREADS) v += a.group_loss[g];
  v = block_sum_d<PREF_MEAN_THREADS>(v, sh);
  if (threadIdx.x == 0) a.loss[0] = (float)(v / (double)a.c.n_group);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int64_t pol_blocks(int64_t n) { return std::max<int64_t>(1, (n + POL_TILE - 1) / POL_TILE); }

template <class E>
hipError_t policy_t(PolArgs& a, void* ws, hipStream_t st) {
  const rece_policy_config& c = a.c;
  if (c.n <= POL_SMALL_N && c.n_seq <= POL_SMALL_SEQ) {
    hipLaunchKernelGGL(k_pol_small<E>, dim3(1), dim3(POL_SMALL_THREADS), 0, st, a);
    return hipGetLastError();
  }
  const int64_t blocks = pol_blocks(c.n);
  const bool per_seq = c.reduction == RECE_MEAN_SEQUENCE;
  a.partial = static_cast<double*>(ws);
  a.part = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + align256((size_t)blocks * 64));
  a.cnt = a.part + 2 * POL_COUNTERS;
  a.counters = per_seq || a.mask ? (int)std::min<int64_t>(blocks, POL_COUNTERS) : 0;
  hipError_t e;
  if (per_seq) {
    hipLaunchKernelGGL(k_pol_clear, dim3((unsigned)((c.n_seq + POL_THREADS - 1) / POL_THREADS)), dim3(POL_THREADS), 0, st,
                       a.cnt, c.n_seq);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.counters) {
    hipLaunchKernelGGL(k_pol_count, dim3((unsigned)a.counters), dim3(POL_THREADS), 0, st, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // four tokens at a time where every array allows it (slices of a longer batch may not): mean over tokens, 65,536 of
  // them 17.8 us against 22.6, a million 19.4 against 24.0, 4.2M 34.9 against 36.0
  uintptr_t tok = 0;
  for (const void* p : {a.logp, a.old, a.ref, a.entropy, static_cast<const void*>(a.dlogp), static_cast<const void*>(a.dentropy)})
    tok |= reinterpret_cast<uintptr_t>(p);
  const bool wide = tok % (4 * sizeof(E)) == 0 && reinterpret_cast<uintptr_t>(a.mask) % 4 == 0;
  auto kern = wide ? k_pol_main<E, 4> : k_pol_main<E, 1>;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(POL_THREADS), 0, st, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pol_final, dim3(1), dim3(POL_THREADS), 0, st, a, blocks);
  return hipGetLastError();
}

template <class E, int L, int W, int NT>
hipError_t pref_launch(const PrefArgs& a, hipStream_t st) {
  const int64_t extra = std::min<int64_t>((a.c.n_seq + NT / L - 1) / (NT / L), PREF_EXTRA);
  const int64_t blocks = a.c.n_group + extra, x = std::min<int64_t>(blocks, 1 << 22);   // at most 2^30 threads along x
  hipLaunchKernelGGL((k_pref<E, L, W, NT>), dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(NT), 0, st, a, (int)extra);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pref_mean, dim3(1), dim3(PREF_MEAN_THREADS), 0, st, a);
  return hipGetLastError();
}

template <class E, int T, int W>
hipError_t pref_many_launch(const PrefArgs& a, hipStream_t st) {
  constexpr int NG = PREF_MANY_THREADS / T;
  const int64_t extra = std::min<int64_t>((a.c.n_seq + NG - 1) / NG, PREF_EXTRA);
  const int64_t blocks = (a.c.n_group + NG - 1) / NG + extra, x = std::min<int64_t>(blocks, 1 << 22);   // at most 2^30 threads along x
  hipLaunchKernelGGL((k_pref_many<E, T, W>), dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(PREF_MANY_THREADS), 0, st, a,
                     (int)extra);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pref_mean, dim3(1), dim3(PREF_MEAN_THREADS), 0, st, a);
  return hipGetLastError();
}

template <class E>
hipError_t preference_t(const PrefArgs& a, hipStream_t st) {
  const int64_t len = a.c.n / a.c.n_seq, group = a.c.n / a.c.n_group;
  const uintptr_t tok = reinterpret_cast<uintptr_t>(a.logp) | reinterpret_cast<uintptr_t>(a.ref) | reinterpret_cast<uintptr_t>(a.dlogp);
  const bool wide = tok % (4 * sizeof(E)) == 0 && reinterpret_cast<uintptr_t>(a.mask) % 4 == 0;
  // Many small groups: a few lanes each, members one after the other, against a workgroup each (us, softmax):
  //   pairs of 1 / 8 / 40 tokens: 1,024 pairs 7.4 / 9.0 / 9.9 against 7.2 / 7.9 / 8.2, 2,048 7.6 / 8.8 / 9.9 against
  //     8.2 / 8.7 / 9.4, 8,192 8.2 / 9.6 / 10.8 against 15.7 / 17.7 / 19.3, 131,072 25 / 48 / 60 against 165 / 189 / 210
  //   groups of 8: 8,192 groups 18 / 27 / 36 against 16 / 18 / 32, 32,768 26 / 35 / 50 against 43 / 52 / 110
  const int64_t G = a.c.n_group;
  if (len < 64 && ((G >= PREF_PAIRS && a.c.n_seq <= 2 * G) || (G > PREF_MANY && a.c.n_seq <= 8 * G))) {
    if (len < 4) return pref_many_launch<E, 1, 1>(a, st);
    return wide ? pref_many_launch<E, 8, 4>(a, st) : pref_many_launch<E, 8, 1>(a, st);
  }
  // Lanes per sequence by the mean length, four tokens each where every array allows it (slices of a longer batch may
  // not).  A million tokens in groups of 16, us with 8 lanes against 1: length 2 60 against 46, 3 43 against 35, 4 33
  // against 29, 8 20 against 21, 16 18 against 21, 32 13 against 18.  A wave takes groups of less than 256 tokens alone.
  if (len >= 64) return wide ? pref_launch<E, 64, 4, 256>(a, st) : pref_launch<E, 64, 1, 256>(a, st);
  if (len < 4) return pref_launch<E, 1, 1, 64>(a, st);
  if (group >= 256) return wide ? pref_launch<E, 8, 4, 256>(a, st) : pref_launch<E, 8, 1, 256>(a, st);
  return wide ? pref_launch<E, 8, 4, 64>(a, st) : pref_launch<E, 8, 1, 64>(a, st);
}

}  // namespace

size_t policy_workspace_bytes(const rece_policy_config& c) {
  if (c.n <= POL_SMALL_N && c.n_seq <= POL_SMALL_SEQ) return 16;
  return align256((size_t)pol_blocks(c.n) * 64) + (size_t)POL_COUNTERS * 8 +
         align256((size_t)(c.reduction == RECE_MEAN_SEQUENCE ? c.n_seq : 0) * 4);
}

hipError_t policy_loss(const rece_policy_config& c, const void* logp, const void* old, const void* ref,
                       const void* entropy, const float* adv, const int32_t* offsets, const uint8_t* mask,
                       const float* dloss, void* ws, float* loss, float* stats, void* dlogp, void* dentropy,
                       hipStream_t st) {
  PolArgs a{};
  a.c = c;
  a.logp = logp;
  a.old = old;
  a.ref = ref;
  a.entropy = entropy;
  a.adv = adv;
  a.offs = offsets;
  a.mask = mask;
  a.dloss = dloss;
  a.loss = loss;
  a.stats = stats;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  // clip_low = 1: a bound of 0 that no ratio is below, so its logarithm is minus infinity, with nothing left
  const double lo = c.clip_low < 1.0f ? std::log1p(-(double)c.clip_low) : -HUGE_VAL, hi = std::log1p((double)c.clip_high);
  a.log_lo = (float)lo;
  a.log_lo2 = c.clip_low < 1.0f ? (float)(lo - (double)a.log_lo) : 0.0f;
  a.log_hi = (float)hi;
  a.log_hi2 = (float)(hi - (double)a.log_hi);
  return c.dtype == RECE_BF16 ? policy_t<bf16>(a, ws, st) : policy_t<float>(a, ws, st);
}

size_t preference_workspace_bytes(const rece_preference_config& c) {
  const size_t groups = align256((size_t)c.n_group * 8);
  if (c.n_seq <= PREF_LDS) return groups;   // every group's members fit into LDS
  return groups + 2 * align256((size_t)c.n_seq * 8);
}

hipError_t preference_loss(const rece_preference_config& c, const void* logp, const void* ref, const int32_t* offsets,
                           const int32_t* group_offsets, const uint8_t* mask, const float* dloss, void* ws, float* loss,
                           float* loss_pg, float* rewards, void* dlogp, hipStream_t st) {
  PrefArgs a{};
  a.c = c;
  a.logp = logp;
  a.ref = ref;
  a.offs = offsets;
  a.goffs = group_offsets;
  a.mask = mask;
  a.dloss = dloss;
  a.group_loss = static_cast<double*>(ws);
  a.h = reinterpret_cast<double*>(static_cast<char*>(ws) + align256((size_t)c.n_group * 8));
  a.share = reinterpret_cast<double*>(static_cast<char*>(ws) + align256((size_t)c.n_group * 8) + align256((size_t)c.n_seq * 8));
  a.loss = loss;
  a.loss_pg = loss_pg;
  a.rewards = rewards;
  a.dlogp = dlogp;
  return c.dtype == RECE_BF16 ? preference_t<bf16>(a, st) : preference_t<float>(a, st);
}

}  // namespace rece
