// Losses on log-probabilities of ragged sequences, with their gradients in the same pass:
// the clipped policy loss with a KL and an entropy term, and the preference loss over
// groups of sequences.  Formulas in include/rece.h.  Both are bound by memory: a token is
// a few floats read and one written, and every token is touched once (the policy loss
// reads the mask a second time, for the number of tokens its mean divides by).
// Sums are taken in float64: they are few beside the bytes, and a float32 sum over
// millions of tokens would lose the small differences these losses are made of.
#include <algorithm>

#include "rece_device.h"
#include "rece_internal.h"

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
constexpr int POL_SMALL_N = 8192;   // one workgroup takes the whole call up to this many tokens ...
constexpr int POL_SMALL_SEQ = 2048; // ... and sequences (their offsets and counts lie in LDS)
constexpr int POL_SUMS = 7;         // loss, pg, kl, entropy, clipped, ratio, tokens

struct PolArgs {
  rece_policy_config c;
  const void *logp, *old, *ref, *entropy;
  const float* adv;
  const int32_t* offs;
  const uint8_t* mask;
  const float* dloss;
  float *loss, *stats;
  void *dlogp, *dentropy;
  int32_t* head;        // [2] tokens that count, sequences with such a token
  int32_t* cnt;         // [n_seq] tokens that count (sequence mean)
  double* partial;      // [blocks][8]
};

struct PolSums {
  double v[POL_SUMS];
};

// One token that counts: its weight w, advantage A; returns the gradients by logp and entropy (without dloss).
template <class E>
__device__ __forceinline__ void pol_token(const PolArgs& a, int64_t t, float w, float A, PolSums& s, float& dlp, float& dent) {
  const float lp = to_f32(static_cast<const E*>(a.logp)[t]);
  const float r = expf(lp - to_f32(static_cast<const E*>(a.old)[t]));
  const float lo = 1.0f - a.c.clip_low, hi = 1.0f + a.c.clip_high;
  const bool clipped = (A > 0.0f && r > hi) || (A < 0.0f && r < lo);
  const float pg = clipped ? -A * (A > 0.0f ? hi : lo) : -A * r;
  float g = clipped ? 0.0f : -A * r;
  float kl = 0.0f, H = 0.0f;
  if (a.ref) {
    const float u = to_f32(static_cast<const E*>(a.ref)[t]) - lp;
    const float eu = expf(u);
    kl = eu - u - 1.0f;
    if (a.c.kl_coef != 0.0f) g = fmaf(a.c.kl_coef, 1.0f - eu, g);
  }
  if (a.entropy) H = to_f32(static_cast<const E*>(a.entropy)[t]);
  // without a coefficient a term is no part of the loss, whatever its value
  float total = pg;
  if (a.c.kl_coef != 0.0f) total = fmaf(a.c.kl_coef, kl, total);
  if (a.c.entropy_coef != 0.0f) total = fmaf(-a.c.entropy_coef, H, total);
  s.v[0] += (double)w * (double)total;
  s.v[1] += pg;
  s.v[2] += kl;
  s.v[3] += H;
  s.v[4] += clipped ? 1.0 : 0.0;
  s.v[5] += r;
  s.v[6] += 1.0;
  dlp = w * g;
  dent = -a.c.entropy_coef * w;
}

__global__ __launch_bounds__(POL_THREADS) void k_pol_clear(int32_t* __restrict__ p, int64_t n) {
  const int64_t t = (int64_t)blockIdx.x * POL_THREADS + threadIdx.x;
  if (t < n) p[t] = 0;
}

// Tokens that count: all (token mean) or per sequence, and the sequences that have one.
__global__ __launch_bounds__(POL_THREADS) void k_pol_count(PolArgs a) {
  constexpr int PER = POL_TILE / POL_THREADS;
  const int64_t n = a.c.n, ns = a.c.n_seq;
  const int64_t base = (int64_t)blockIdx.x * POL_TILE, t0 = base + (int64_t)threadIdx.x * PER;
  const int64_t lo = max(offset_at(a.offs, 0, n), t0), hi = min(offset_at(a.offs, ns, n), min(n, t0 + PER));
  const bool per_seq = a.c.reduction == RECE_MEAN_SEQUENCE;
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
  if (!per_seq) {
    const int c = wave_sum(__popc(bits));
    if (lane_id() == 0 && c) atomicAdd(&a.head[0], c);   // integers: any order gives the same sum
    return;
  }
  const int64_t wave0 = base + (int64_t)(threadIdx.x & ~(WAVE - 1)) * PER;
  if (wave0 >= n) return;   // whole waves
  const int64_t s0 = seq_of_wave(a.offs, 0, ns - 1, wave0);
  const int64_t s1 = seq_of_wave(a.offs, s0, ns - 1, min(n, wave0 + WAVE * PER) - 1);
  auto add = [&](int64_t s, int c) {
    if (atomicAdd(&a.cnt[s], c) == 0) atomicAdd(&a.head[1], 1);
  };
  if (s0 == s1) {
    const int c = wave_sum(__popc(bits));
    if (lane_id() == 0 && c) add(s0, c);
    return;
  }
  int64_t t = lo;
  while (t < hi) {
    const int64_t s = seq_of(a.offs, s0, s1, t);
    const int64_t e = max(t + 1, min(hi, s + 1 <= ns ? offset_at(a.offs, s + 1, n) : hi));
    const uint32_t part = bits & ~((1u << (t - t0)) - 1u) & (e - t0 >= 32 ? ~0u : (1u << (e - t0)) - 1u);
    if (part) add(s, __popc(part));
    t = e;
  }
}

template <class E>
__global__ __launch_bounds__(POL_THREADS) void k_pol_main(PolArgs a) {
  __shared__ double sh[POL_THREADS / WAVE];
  const int64_t n = a.c.n, ns = a.c.n_seq;
  const int64_t lo = offset_at(a.offs, 0, n), hi = offset_at(a.offs, ns, n);
  const int64_t base = (int64_t)blockIdx.x * POL_TILE;
  const bool per_seq = a.c.reduction == RECE_MEAN_SEQUENCE, need_seq = per_seq || !a.c.token_adv;
  const int64_t tokens = a.head ? (int64_t)a.head[0] : hi - lo;
  const float up = a.dloss ? a.dloss[0] : 1.0f;
  const float wt = 1.0f / (float)max(tokens, (int64_t)1);
  const float nonempty = per_seq ? (float)max(a.head[1], 1) : 1.0f;
  PolSums s{};
  int64_t s0 = 0, s1 = 0;
  if (need_seq) {
    s0 = seq_of_wave(a.offs, 0, ns - 1, base);
    s1 = seq_of_wave(a.offs, s0, ns - 1, min(n, base + POL_TILE) - 1);
  }
  for (int q = 0; q < POL_TILE / POL_THREADS; ++q) {
    const int64_t t = base + q * POL_THREADS + threadIdx.x;
    if (t >= n) break;
    float dlp = 0.0f, dent = 0.0f;
    if (t >= lo && t < hi && (!a.mask || a.mask[t])) {
      const int64_t sq = need_seq ? seq_of(a.offs, s0, s1, t) : 0;
      const float w = per_seq ? 1.0f / ((float)max(a.cnt[sq], 1) * nonempty) : wt;
      pol_token<E>(a, t, w, a.adv[a.c.token_adv ? t : sq], s, dlp, dent);
    }
    if (a.dlogp) put(static_cast<E*>(a.dlogp), t, up * dlp);
    if (a.dentropy) put(static_cast<E*>(a.dentropy), t, up * dent);
  }
#pragma unroll
  for (int k = 0; k < POL_SUMS; ++k) {
    const double v = block_sum_d<POL_THREADS>(s.v[k], sh);
    if (threadIdx.x == 0) a.partial[(int64_t)blockIdx.x * 8 + k] = v;
  }
}

__device__ __forceinline__ void pol_write(const PolArgs& a, const double (&v)[POL_SUMS]) {
  const double m = v[6] > 0.0 ? 1.0 / v[6] : 0.0;
  a.loss[0] = (float)v[0];
#pragma unroll
  for (int k = 1; k < 6; ++k) a.stats[k - 1] = (float)(v[k] * m);
  a.stats[5] = (float)v[6];
}

__global__ __launch_bounds__(POL_THREADS) void k_pol_final(PolArgs a, int64_t blocks) {
  __shared__ double sh[POL_THREADS / WAVE];
  double v[POL_SUMS];
#pragma unroll
  for (int k = 0; k < POL_SUMS; ++k) v[k] = 0.0;
  for (int64_t b = threadIdx.x; b < blocks; b += POL_THREADS)
#pragma unroll
    for (int k = 0; k < POL_SUMS; ++k) v[k] += a.partial[b * 8 + k];
#pragma unroll
  for (int k = 0; k < POL_SUMS; ++k) v[k] = block_sum_d<POL_THREADS>(v[k], sh);
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
  const int n = (int)a.c.n, ns = (int)a.c.n_seq;
  const bool per_seq = a.c.reduction == RECE_MEAN_SEQUENCE;
  for (int i = threadIdx.x; i <= ns; i += POL_SMALL_THREADS) {
    offs[i] = (int32_t)offset_at(a.offs, i, n);
    if (i < ns) cnt[i] = 0;
  }
  __syncthreads();
  int sq[PER];
  int mine = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int t = q * POL_SMALL_THREADS + (int)threadIdx.x;
    sq[q] = -1;
    if (t >= offs[0] && t < offs[ns] && (!a.mask || a.mask[t])) {
      int lo = 0, hi = ns - 1;
      while (lo < hi) {
        const int m = (lo + hi + 1) / 2;
        if (offs[m] <= t) lo = m; else hi = m - 1;
      }
      sq[q] = lo;
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
  const float wt = 1.0f / (float)fmax(tokens, 1.0), nonempty = (float)fmax(with, 1.0);
  const float up = a.dloss ? a.dloss[0] : 1.0f;
  PolSums s{};
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int t = q * POL_SMALL_THREADS + (int)threadIdx.x;
    if (t >= n) break;
    float dlp = 0.0f, dent = 0.0f;
    if (sq[q] >= 0) {
      const float w = per_seq ? 1.0f / ((float)cnt[sq[q]] * nonempty) : wt;
      pol_token<E>(a, t, w, a.adv[a.c.token_adv ? t : sq[q]], s, dlp, dent);
    }
    if (a.dlogp) put(static_cast<E*>(a.dlogp), t, up * dlp);
    if (a.dentropy) put(static_cast<E*>(a.dentropy), t, up * dent);
  }
  double v[POL_SUMS];
#pragma unroll
  for (int k = 0; k < POL_SUMS; ++k) v[k] = block_sum_d<POL_SMALL_THREADS>(s.v[k], sh);
  if (threadIdx.x == 0) pol_write(a, v);
}

// ------------------------------------------------------------------ preference loss
struct PrefArgs {
  rece_preference_config c;
  const void *logp, *ref;
  const int32_t *offs, *goffs;
  const uint8_t* mask;
  const float* dloss;
  double* h;            // [n_seq]
  float* share;         // [n_seq] 1, or 1 / tokens that count (average)
  float *loss, *loss_pg, *rewards;
  void* dlogp;
};

// h of sequence i by L lanes (all of them get it).
template <class E, int L>
__device__ __forceinline__ double pref_sum(const PrefArgs& a, int64_t i, int sub, float& share) {
  const int64_t lo = offset_at(a.offs, i, a.c.n), hi = max(lo, offset_at(a.offs, i + 1, a.c.n));
  const E* lp = static_cast<const E*>(a.logp);
  const E* rf = static_cast<const E*>(a.ref);
  double s = 0.0;
  int c = 0;
  for (int64_t t = lo + sub; t < hi; t += L) {
    if (a.mask && !a.mask[t]) continue;
    s += (double)(rf ? to_f32(lp[t]) - to_f32(rf[t]) : to_f32(lp[t]));
    ++c;
  }
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) {
    s += __shfl_xor(s, o);
    c += __shfl_xor(c, o);
  }
  share = a.c.average ? 1.0f / (float)max(c, 1) : 1.0f;
  return a.c.average ? s / (double)max(c, 1) : s;
}

// Gradient of sequence i's tokens: v where they count, else 0.
template <class E, int L>
__device__ __forceinline__ void pref_grad(const PrefArgs& a, int64_t i, int sub, float v) {
  const int64_t lo = offset_at(a.offs, i, a.c.n), hi = max(lo, offset_at(a.offs, i + 1, a.c.n));
  for (int64_t t = lo + sub; t < hi; t += L) put(static_cast<E*>(a.dlogp), t, a.mask && !a.mask[t] ? 0.0f : v);
}

__device__ __forceinline__ double softplus_d(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

// Loss of one pair and its derivative by z.
__device__ __forceinline__ double pair_loss(const rece_preference_config& c, double z, double& dz) {
  if (c.kind == RECE_PREF_SIGMOID) {
    const double e = c.smoothing;
    dz = 1.0 / (1.0 + exp(-z)) - (1.0 - e);
    return (1.0 - e) * softplus_d(-z) + e * softplus_d(z);
  }
  if (c.kind == RECE_PREF_IPO) {
    const double b = c.beta, v = z / b - 0.5 / b;
    dz = 2.0 * v / b;
    return v * v;
  }
  dz = z < 1.0 ? -1.0 : 0.0;
  return fmax(0.0, 1.0 - z);
}

constexpr int PREF_LDS = 512;   // sequences of a group whose h lies in LDS

// Workgroups 0 .. n_group - 1: one group each.  The others: the sequences in no group, and
// the tokens in no sequence.
template <class E, int L, int NT>
__global__ __launch_bounds__(NT) void k_pref(PrefArgs a) {
  constexpr int NS = NT / L;   // sequences at a time
  __shared__ double sh_h[PREF_LDS];
  __shared__ float sh_share[PREF_LDS];
  const int64_t G = a.c.n_group, nseq = a.c.n_seq;
  const int q = threadIdx.x / L, sub = threadIdx.x % L;
  const float beta = a.c.beta;
  if ((int64_t)blockIdx.x >= G) {
    const int64_t first = offset_at(a.goffs, 0, nseq), end = offset_at(a.goffs, G, nseq);
    const int64_t extra = (int64_t)gridDim.x - G, b = (int64_t)blockIdx.x - G;
    for (int64_t k = b * NS + q; k < first + (nseq - end); k += extra * NS) {
      const int64_t i = k < first ? k : end + (k - first);
      if (i >= nseq) break;
      float share;
      const double h = pref_sum<E, L>(a, i, sub, share);
      if (sub == 0) a.rewards[i] = (float)((double)beta * h);
      if (a.dlogp) pref_grad<E, L>(a, i, sub, 0.0f);
    }
    if (a.dlogp) {
      const int64_t lo = offset_at(a.offs, 0, a.c.n), hi = max(lo, offset_at(a.offs, nseq, a.c.n));
      for (int64_t k = b * NT + threadIdx.x; k < lo + (a.c.n - hi); k += extra * NT)
        put(static_cast<E*>(a.dlogp), k < lo ? k : hi + (k - lo), 0.0f);
    }
    return;
  }
  const int64_t g = blockIdx.x;
  const int64_t s0 = offset_at(a.goffs, g, nseq), s1 = max(s0, offset_at(a.goffs, g + 1, nseq));
  const int64_t m = s1 - s0;
  const bool in_lds = m <= PREF_LDS;
  for (int64_t k = q; k < m; k += NS) {
    float share;
    const double h = pref_sum<E, L>(a, s0 + k, sub, share);
    if (sub == 0) {
      a.rewards[s0 + k] = (float)((double)beta * h);
      if (in_lds) {
        sh_h[k] = h;
        sh_share[k] = share;
      } else {
        a.h[s0 + k] = h;
        a.share[s0 + k] = share;
      }
    }
  }
  __syncthreads();
  auto h_at = [&](int64_t k) { return in_lds ? sh_h[k] : a.h[s0 + k]; };
  auto share_at = [&](int64_t k) { return in_lds ? sh_share[k] : a.share[s0 + k]; };
  // every wave takes the group's loss by itself
  const int l = lane_id();
  const bool soft = a.c.kind == RECE_PREF_SOFTMAX;
  double loss = 0.0, dc = 0.0, top = 0.0, tot = 1.0, per = 0.0;
  if (m >= 2) {
    const double hc = h_at(0);
    auto z_of = [&](int64_t k) { return (double)beta * (hc - h_at(k)) - (double)a.c.margin; };
    per = 1.0 / (double)(m - 1);
    if (soft) {
      for (int64_t k = 1 + l; k < m; k += WAVE) top = fmax(top, -z_of(k));
      top = wave_max_d(top);
      tot = 0.0;
      for (int64_t k = 1 + l; k < m; k += WAVE) tot += exp(-z_of(k) - top);
      const double others = wave_sum_d(tot);
      tot = others + exp(-top);
      loss = top + log(tot);
      dc = -others / tot;
    } else {
      for (int64_t k = 1 + l; k < m; k += WAVE) {
        double dz;
        loss += pair_loss(a.c, z_of(k), dz);
        dc += dz;
      }
      loss = wave_sum_d(loss) * per;
      dc = wave_sum_d(dc) * per;
    }
  }
  if (threadIdx.x == 0) a.loss_pg[g] = (float)loss;
  if (!a.dlogp) return;
  const double up = (double)beta * (a.dloss ? (double)a.dloss[0] : 1.0) / (double)G;
  for (int64_t k = q; k < m; k += NS) {
    double dh = dc;
    if (k > 0) {
      const double z = (double)beta * (h_at(0) - h_at(k)) - (double)a.c.margin;
      if (soft) {
        dh = exp(-z - top) / tot;
      } else {
        double dz;
        pair_loss(a.c, z, dz);
        dh = -dz * per;
      }
    }
    pref_grad<E, L>(a, s0 + k, sub, (float)(dh * up * (double)share_at(k)));
  }
}

__global__ __launch_bounds__(256) void k_pref_mean(PrefArgs a) {
  __shared__ double sh[256 / WAVE];
  double v = 0.0;
  for (int64_t g = threadIdx.x; g < a.c.n_group; g += 256) v += a.loss_pg[g];
  v = block_sum_d<256>(v, sh);
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
  if (per_seq || a.mask) {   // else the number of tokens is known from the offsets
    a.head = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + align256((size_t)blocks * 64));
    a.cnt = a.head + 2;
    const int64_t words = 2 + (per_seq ? c.n_seq : 0);
    hipLaunchKernelGGL(k_pol_clear, dim3((unsigned)((words + POL_THREADS - 1) / POL_THREADS)), dim3(POL_THREADS), 0, st,
                       a.head, words);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_pol_count, dim3((unsigned)blocks), dim3(POL_THREADS), 0, st, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_pol_main<E>, dim3((unsigned)blocks), dim3(POL_THREADS), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pol_final, dim3(1), dim3(POL_THREADS), 0, st, a, blocks);
  return hipGetLastError();
}

template <class E, int L, int NT>
hipError_t pref_launch(const PrefArgs& a, hipStream_t st) {
  const int64_t extra = std::min<int64_t>((a.c.n_seq + NT / L - 1) / (NT / L), 1024);
  hipLaunchKernelGGL((k_pref<E, L, NT>), dim3((unsigned)(a.c.n_group + extra)), dim3(NT), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pref_mean, dim3(1), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <class E>
hipError_t preference_t(const PrefArgs& a, hipStream_t st) {
  const int64_t len = a.c.n / a.c.n_seq, group = a.c.n / a.c.n_group;
  if (len >= 32) return pref_launch<E, 64, 256>(a, st);
  if (len >= 4 && group >= 256) return pref_launch<E, 8, 256>(a, st);
  if (len >= 4) return pref_launch<E, 8, 64>(a, st);
  return pref_launch<E, 1, 64>(a, st);
}

}  // namespace

size_t policy_workspace_bytes(const rece_policy_config& c) {
  if (c.n <= POL_SMALL_N && c.n_seq <= POL_SMALL_SEQ) return 16;
  return align256((size_t)pol_blocks(c.n) * 64) +
         align256((size_t)(2 + (c.reduction == RECE_MEAN_SEQUENCE ? c.n_seq : 0)) * 4);
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
  return c.dtype == RECE_BF16 ? policy_t<bf16>(a, ws, st) : policy_t<float>(a, ws, st);
}

size_t preference_workspace_bytes(const rece_preference_config& c) {
  return align256((size_t)c.n_seq * 8) + align256((size_t)c.n_seq * 4);
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
  a.h = static_cast<double*>(ws);
  a.share = reinterpret_cast<float*>(static_cast<char*>(ws) + align256((size_t)c.n_seq * 8));
  a.loss = loss;
  a.loss_pg = loss_pg;
  a.rewards = rewards;
  a.dlogp = dlogp;
  return c.dtype == RECE_BF16 ? preference_t<bf16>(a, st) : preference_t<float>(a, st);
}

}  // namespace rece
