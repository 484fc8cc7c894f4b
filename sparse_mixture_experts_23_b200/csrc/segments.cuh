// Expert segments of row-grouped operands, read from a caller's offsets array.
#pragma once
#include <stdint.h>

#include "moe_internal.cuh"

namespace moe {

constexpr int kMaxExperts = 256;

struct TileCount {  // tiles of a segment of rows
  int tile, per_tile;
  __device__ __forceinline__ int operator()(int rows) const { return (int)(((unsigned)rows + tile - 1) / (unsigned)tile) * per_tile; }
};

template <int PER, typename Cost>
__device__ __forceinline__ void load_segments_impl(const int32_t* __restrict__ in, int E, int cap, Cost cost, int* offs,
                                                   int* prefix, int32_t* status, bool report) {
  const int lane = threadIdx.x & 31;
  int raw[PER], v[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) raw[j] = lane * PER + j <= E ? in[lane * PER + j] : 0;
  bool bad = false;
  int run = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = lane * PER + j;
    int c = raw[j] < 0 ? 0 : (raw[j] > cap ? cap : raw[j]);
    if (i == 0) c = 0;
    if (c != raw[j]) bad = true;
    if (i <= E && c < run) bad = true;
    run = max(run, c);
    v[j] = run;
  }
  int before = run;  // inclusive maximum over lanes, then the one of the lanes below
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before = max(before, u);
  }
  before = __shfl_up_sync(0xffffffffu, before, 1);
  if (lane == 0) before = 0;
  if (lane * PER <= E && v[0] < before) bad = true;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = lane * PER + j;
    v[j] = max(v[j], before);
    if (i <= E) offs[i] = v[j];
  }
  if (report && status != nullptr && __any_sync(0xffffffffu, bad) && lane == 0) atomicCAS(status, 0, kDevBadIndex);
  if (prefix == nullptr) {
    __syncwarp();
    return;
  }
  const int next_first = __shfl_down_sync(0xffffffffu, v[0], 1);
  int t[PER], sum = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = lane * PER + j;
    const int hi = j + 1 < PER ? v[j + 1 < PER ? j + 1 : j] : next_first;
    t[j] = sum;
    if (i < E) sum += cost(hi - v[j]);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  const int excl = incl - sum;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = lane * PER + j;
    if (i <= E) prefix[i] = excl + t[j];
  }
  __syncwarp();
}

// Called by one full warp.  offs[0..E] = the caller's offsets made safe to index with (from 0,
// non-decreasing, at most rows_cap), prefix[e] = sum over experts before e of cost(rows) (prefix may be
// null).  A changed entry is recorded in the optional error word by the caller whose report is true.
// Each lane takes 9 entries in a row (one where 32 hold them all: every kernel waits for this at its
// start); running maxima and sums are joined by shuffles, so 257 entries cost two short scans instead of
// one thread's 257 dependent steps.
template <typename Cost>
__device__ __forceinline__ void load_segments(const int32_t* __restrict__ in, int E, long long rows_cap, Cost cost, int* offs,
                                              int* prefix, int32_t* status, bool report) {
  static_assert(32 * 9 >= kMaxExperts + 1, "one warp covers every expert");
  const int cap = rows_cap > 0x7fffffffLL ? 0x7fffffff : (int)rows_cap;
  if (E < 32) load_segments_impl<1>(in, E, cap, cost, offs, prefix, status, report);
  else load_segments_impl<9>(in, E, cap, cost, offs, prefix, status, report);
}
// prefix[e] counts tiles: ceil(rows / tile) * per_tile each
__device__ __forceinline__ void load_segments(const int32_t* __restrict__ in, int E, long long rows_cap, int tile,
                                              int per_tile, int* offs, int* prefix, int32_t* status, bool report) {
  load_segments(in, E, rows_cap, TileCount{tile, per_tile}, offs, prefix, status, report);
}

// The last expert whose first tile is not past `tile` (experts without tiles are skipped).
__device__ __forceinline__ int find_segment(const int* prefix, int E, int tile) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace moe
