// How a sweep's work is dealt to workgroups, and where its partial results lie.
//
// The units (owner block b, tile t of the streamed side), b major, are cut into equal runs of
// `per` units, one workgroup g each, so every workgroup does the same work whatever the number of
// owner blocks; a run may end inside an owner block.  Workgroup g's part of block b lies in slot b + g
// (the pairs that occur form a staircase, so the slots are distinct and at most blocks + workgroups).
// With `whole`, the runs are rounded up to whole owner blocks: block b has one part, in slot b.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rece {

// a / b, by 32-bit division where both fit (a 64-bit one costs several times as much).
__device__ __forceinline__ uint64_t div_u64(uint64_t a, uint64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct SweepWork {
  uint32_t nb, nt;   // owner blocks, tiles
  uint64_t total, per;
  bool whole;
  // where workgroup g's part of block b lies
  __device__ __forceinline__ int64_t slot(int64_t b, int64_t g) const { return whole ? b : b + g; }
  // workgroups that hold parts of block b (first > last: none)
  __device__ __forceinline__ int64_t first(uint64_t b) const { return nt == 0 ? 1 : (int64_t)div_u64(b * nt, per); }
  __device__ __forceinline__ int64_t last(uint64_t b) const { return nt == 0 ? 0 : (int64_t)div_u64((b + 1) * nt - 1, per); }
};

struct SweepParts {
  const int32_t* nv;      // packed positions
  int64_t n_own, n_str;   // upper bounds; the positions' side is *nv
  int own_is_pos;         // the owners are the positions (else the streamed side is)
  uint32_t block, tile;   // owners of a block, rows of a tile
  uint32_t grid;          // workgroups
  int nws;                // parts of a workgroup (waves along a tile)
  int whole;              // whole owner blocks per workgroup
  const float* rows;      // [slots][nws][block][d] partial rows
  __device__ __forceinline__ uint32_t owners() const { return own_is_pos ? (uint32_t)*nv : (uint32_t)n_own; }
  __device__ __forceinline__ uint32_t streamed() const { return own_is_pos ? (uint32_t)n_str : (uint32_t)*nv; }
  __device__ __forceinline__ SweepWork work() const {
    SweepWork w;
    w.nb = (uint32_t)div_u64((uint64_t)owners() + block - 1, block);
    w.nt = (uint32_t)div_u64((uint64_t)streamed() + tile - 1, tile);
    w.total = (uint64_t)w.nb * w.nt;
    w.per = whole ? (uint64_t)div_u64((uint64_t)w.nb + grid - 1, grid) * w.nt : div_u64(w.total + grid - 1, grid);
    if (w.per == 0) w.per = 1;
    w.whole = whole != 0;
    return w;
  }
  // f(index of a partial result) for every step-th part of row r from the begin-th on, in order; results are
  // indexed [slots][nws][block].
  template <class F>
  __device__ __forceinline__ void each(const SweepWork& w, int64_t r, F f, int begin = 0, int step = 1) const {
    const uint32_t b = (uint32_t)r / block, at = (uint32_t)r % block;
    const int64_t g0 = w.first(b), g1 = w.last(b);
    const int q0 = (int)w.slot(b, g0) * nws, q1 = g0 <= g1 ? (int)(w.slot(b, g1) + 1) * nws : q0;
#pragma unroll 4
    for (int q = q0 + begin; q < q1; q += step) f((int64_t)q * block + at);
  }
};

}  // namespace rece
