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

constexpr int kGM = 128;              // tile rows (MMA M)

// The kernels count units in 32 bits; more than that many would write more
// than any GPU's memory.
inline bool units_fit(const MmArgs& m, int64_t row_tiles, int64_t n_tiles) {
  return (row_tiles + m.G) * n_tiles * m.S < (1ll << 31) - 4096;
}

// C columns (a multiple of 8) of a row from fp32 bits: n valid ones at p, as
// out_dtype; vec: 16-byte stores are aligned.
template <int C>
__device__ __forceinline__ void store_cols(void* p, const uint32_t (&v)[C], int n, int out_dtype, bool vec) {
  if (out_dtype == MOE_DT_F32) {
    uint32_t* d = reinterpret_cast<uint32_t*>(p);
    if (vec && n >= C) {
#pragma unroll
      for (int i = 0; i < C / 4; ++i)
        reinterpret_cast<uint4*>(d)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < n) d[i] = v[i];
    }
    return;
  }
  uint32_t pk[C / 2];
#pragma unroll
  for (int i = 0; i < C / 2; ++i) {
    const float a = __uint_as_float(v[2 * i]), b = __uint_as_float(v[2 * i + 1]);
    pk[i] = out_dtype == MOE_DT_F16 ? F16::from2(a, b) : Bf16::from2(a, b);
  }
  if (vec && n >= C) {
#pragma unroll
    for (int i = 0; i < C / 8; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
  } else {
    uint16_t* d = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) d[i] = (uint16_t)(pk[i >> 1] >> (16 * (i & 1)));
  }
}

// A warp's 32 rows (lane = row), NU units of 16 bytes each, to row-major out. A
// lane's own row would make every store touch 32 lines; instead the units are
// exchanged among NU lanes (a transpose in log2 NU steps), so that a store
// covers whole segments of 16 NU bytes of 32 / NU rows. p: the first row's
// first unit (16-byte aligned, as row_bytes is); rows < n_rows are written.
template <int NU>
__device__ __forceinline__ void store_units(uint8_t* p, int64_t row_bytes, uint32_t (&w)[NU][4], int n_rows, int lane) {
#pragma unroll
  for (int s = 1; s < NU; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (i & s) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t got = __shfl_xor_sync(kFull, up ? w[i][j] : w[i | s][j], s);
        w[i][j] = up ? got : w[i][j];
        w[i | s][j] = up ? w[i | s][j] : got;
      }
    }
  }
  const int r0 = lane & ~(NU - 1);
  uint8_t* d = p + r0 * row_bytes + (lane & (NU - 1)) * 16;
#pragma unroll
  for (int i = 0; i < NU; ++i)
    if (r0 + i < n_rows) *reinterpret_cast<uint4*>(d + i * row_bytes) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
}
// C columns of those rows from fp32, as out_dtype.
template <int C>
__device__ __forceinline__ void store_block(uint8_t* p, int64_t row_bytes, const float (&v)[C], int n_rows, int lane,
                                            int out_dtype) {
  if (out_dtype == MOE_DT_F32) {
    constexpr int CF = C < 32 ? C : 32;       // 128 bytes a row at a time
#pragma unroll
    for (int k = 0; k < C; k += CF) {
      uint32_t w[CF / 4][4];
#pragma unroll
      for (int i = 0; i < CF; ++i) w[i / 4][i & 3] = __float_as_uint(v[k + i]);
      store_units<CF / 4>(p + 4 * k, row_bytes, w, n_rows, lane);
    }
  } else {
    uint32_t w[C / 8][4];
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
      w[i / 4][i & 3] = out_dtype == MOE_DT_F16 ? F16::from2(v[2 * i], v[2 * i + 1]) : Bf16::from2(v[2 * i], v[2 * i + 1]);
    store_units<C / 8>(p, row_bytes, w, n_rows, lane);
  }
}

// Rows outside every group become zeros (their partial sums, where the product
// is split). One warp of each CTA.
__device__ __forceinline__ void clear_rows_outside(const MmArgs& m, const int32_t* off, int lane) {
  const int lo = off[0], hi = off[m.G];
  for (int64_t r = blockIdx.x; r < m.R - (int64_t)(hi - lo); r += gridDim.x) {
    const int64_t row = r < lo ? r : r - lo + hi;
    if (m.S > 1) {
      for (int s = 0; s < m.S; ++s)
        for (int64_t i = lane; i < m.N; i += 32) m.part[((int64_t)s * m.R + row) * m.N + i] = 0.f;
    } else {
      for (int64_t i = lane; i < m.N; i += 32) {
        if (m.out_dtype == MOE_DT_F32) reinterpret_cast<float*>(m.out)[row * m.ldo + i] = 0.f;
        else reinterpret_cast<uint16_t*>(m.out)[row * m.ldo + i] = 0;
      }
    }
  }
}

}  // namespace moe
