// The table of a ragged product's groups, built by every CTA in shared memory
// from the device offsets.
#pragma once
#include "ops.cuh"

namespace moe {

constexpr int kMmMaxGroups = 2048;

// off[e] (e <= G): first row of group e, clamped so that 0 <= off[0] <= ... <=
// off[G] <= R whatever the caller's array holds (a change sets
// MOE_DEV_BAD_OFFSETS); offsets == nullptr: one group of all rows. uoff[e]:
// units of the groups before e, where a group of c rows has tiles(c) of them.
// Called by all THREADS threads; `tmp` holds 2 * THREADS / 32 ints. Ends with a
// barrier.
template <int THREADS, typename Tiles>
__device__ __forceinline__ void build_groups(const int32_t* offsets, int G, int R, int32_t* off, int32_t* uoff,
                                             int* tmp, int32_t* status, Tiles tiles) {
  constexpr int kPer = (kMmMaxGroups + 1 + THREADS - 1) / THREADS;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // thread t owns entries [t * per, (t + 1) * per) of off[0 .. G]
  const int per = (G + 1 + THREADS - 1) / THREADS, e0 = t * per;
  int v[kPer];
  int run = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = 0;
    if (i < per && e0 + i <= G) {
      const int e = e0 + i;
      const int raw = offsets ? offsets[e] : (e == 0 ? 0 : R);
      v[i] = min(max(raw, 0), R);
      bad |= v[i] != raw;
      bad |= v[i] < run;
      run = max(run, v[i]);
    }
  }
  // running maximum over the threads before this one
  int mx = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int q = __shfl_up_sync(kFull, mx, o);
    if (lane >= o) mx = max(mx, q);
  }
  if (lane == 31) tmp[warp] = mx;
  int before = __shfl_up_sync(kFull, mx, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  for (int i = 0; i < warp; ++i) before = max(before, tmp[i]);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < per && e0 + i <= G) {
      bad |= v[i] < before;
      before = max(before, v[i]);
      off[e0 + i] = before;
    }
  }
  if (bad && blockIdx.x == 0) set_status(status, MOE_DEV_BAD_OFFSETS);
  __syncthreads();
  // units: exclusive prefix sums of tiles(rows) over e < G, the total at G
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < per && e0 + i < G) {
      v[i] = tiles(off[e0 + i + 1] - off[e0 + i]);
      sum += v[i];
    }
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int q = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += q;
  }
  int* tmp2 = tmp + THREADS / 32;
  if (lane == 31) tmp2[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int i = 0; i < warp; ++i) base += tmp2[i];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < per && e0 + i <= G) {
      uoff[e0 + i] = base;
      if (e0 + i < G) base += v[i];
    }
  }
  __syncthreads();
}

// The group of unit u: the last e with uoff[e] <= u (u < uoff[G]).
__device__ __forceinline__ int group_of_unit(const int32_t* uoff, int G, int u) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (uoff[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace moe
