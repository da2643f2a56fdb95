// Layer norm of rows, forward and backward, for the block the routed layer
// sits in (the norm in front of the router).
//
//   mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps)
//   y  = (x - mu) r gamma + beta
//   xh = (x - mu) r, t = dy gamma
//   dx = r (t - mean(t) - xh mean(t xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound: HBM. A row is read once and kept in registers (packed as it came),
// so the variance is taken about the finished mean, in fp32, without a second
// read. A row belongs to TPR threads of one CTA (a warp for short rows), each
// with NV packs of 16 bytes; a persistent grid walks the rows. The backward's
// threads own the same columns in every row, so the sums over rows of the
// weight's gradient stay in registers and reach memory once per CTA, as fp32
// partial rows that a second kernel adds in a fixed order: no atomics, the
// same bits every run. Where that leaves too few bytes in flight a ring of rows
// in shared memory runs ahead (k_norm_ring).
// Measured, bf16: forward 16384 x 2880 47 us (4.0 TB/s), x 7168 87 (5.4 TB/s),
// 1 x 7168 3.5 us; backward with both weight gradients 16384 x 2880 65 us
// (4.3 TB/s), x 7168 143 (4.9 TB/s). At odd alignments 16384 x 2881 76 and 101
// us. What is left: a row's reductions are two rounds (backward one) of shuffles
// and a barrier, and the few rows an SM has in flight wait for them.
#include "ops.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kNormMaxThreads = 1024;
constexpr int kWarpRowThreads = 256;    // a CTA of warps that hold a row each
constexpr int kNormBwdThreads = 512;    // the backward holds four fp32 or packed values a column

// Sums of a and b over the threads of a row (BLOCK: the nw warps of the CTA,
// else the warp), in a fixed order, known to all of them. The first step of
// each round sends one sum to the lower and one to the upper half-warp, so
// two sums take five shuffles, not ten; the warps' sums cross shared memory
// (red: one float2 a warp) behind one barrier. Consecutive calls alternate
// between two buffers.
template <bool BLOCK>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red, int nw) {
  const int lane = threadIdx.x & 31;
  const bool up = lane & 16;
  float v = (up ? b : a) + __shfl_xor_sync(kFull, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if constexpr (BLOCK) {
    float* mine = reinterpret_cast<float*>(red + (threadIdx.x >> 5)) + (up ? 1 : 0);
    if ((lane & 15) == 0) *mine = v;
    __syncthreads();
    const float* r = reinterpret_cast<const float*>(red) + (up ? 1 : 0);
    const int i = lane & 15;
    v = i < nw ? r[2 * i] : 0.f;
    if (nw > 16) v += i + 16 < nw ? r[2 * (i + 16)] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  }
  return make_float2(__shfl_sync(kFull, v, 0), __shfl_sync(kFull, v, 16));
}
// Four sums over a CTA of at most 16 warps, as row_sum2 (red: a float4 a warp).
__device__ __forceinline__ float4 row_sum4(float a, float b, float c, float d, float4* red, int nw) {
  const int lane = threadIdx.x & 31;
  const bool u16 = lane & 16, u8 = lane & 8;
  float v = (u16 ? c : a) + __shfl_xor_sync(kFull, u16 ? a : c, 16);      // a, b below; c, d above
  float w = (u16 ? d : b) + __shfl_xor_sync(kFull, u16 ? b : d, 16);
  v = (u8 ? w : v) + __shfl_xor_sync(kFull, u8 ? v : w, 8);               // lane / 8: a, b, c, d
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  const int k = lane >> 3, i = lane & 7;
  float* mine = reinterpret_cast<float*>(red + (threadIdx.x >> 5)) + k;
  if (i == 0) *mine = v;
  __syncthreads();
  const float* r = reinterpret_cast<const float*>(red) + k;
  v = i < nw ? r[4 * i] : 0.f;
  if (nw > 8) v += i + 8 < nw ? r[4 * (i + 8)] : 0.f;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return make_float4(__shfl_sync(kFull, v, 0), __shfl_sync(kFull, v, 8), __shfl_sync(kFull, v, 16),
                     __shfl_sync(kFull, v, 24));
}
// One sum.
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float a, float2* red, int nw) {
  a = warp_sum(a);
  if constexpr (BLOCK) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5].x = a;
    __syncthreads();
    a = warp_sum(lane < nw ? red[lane].x : 0.f);
  }
  return a;
}

// Element i of a weight vector held in E's type or fp32; `def` when absent.
template <typename E, bool WF32>
__device__ __forceinline__ float weight_at(const void* w, int i, float def) {
  if (!w) return def;
  if constexpr (WF32) return reinterpret_cast<const float*>(w)[i];
  else return E::to(reinterpret_cast<const typename E::raw*>(w)[i]);
}

// V consecutive weights from column c (16-byte accesses where V > 1).
template <typename E, bool WF32, int V>
__device__ __forceinline__ void weights_at(float (&o)[V], const void* w, int c, float def) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = def;
    return;
  }
  if constexpr (V == 1) {
    o[0] = weight_at<E, WF32>(w, c, def);
  } else if constexpr (WF32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + c);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const float4 f = p[j];
      o[4 * j] = f.x; o[4 * j + 1] = f.y; o[4 * j + 2] = f.z; o[4 * j + 3] = f.w;
    }
  } else {
    Pack<E, V> p;
    load_pack(p, reinterpret_cast<const typename E::raw*>(w) + c);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = E::to(p.v[j]);
  }
}

// A pack of a row (VEC: on 16 bytes and whole; else at any alignment, with
// zeros from the row's end on), and its store.
template <typename E, int V, bool VEC>
__device__ __forceinline__ void load_row_pack(Pack<E, V>& p, const typename E::raw* row, int c, int H) {
  if constexpr (VEC) {
    load_pack(p, row + c);
  } else {
    uint32_t w[4];
    load_any<(int)sizeof(typename E::raw), 16>(w, row + c, row, row + H);
    *reinterpret_cast<uint4*>(&p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename E, int V, bool VEC>
__device__ __forceinline__ void store_row_pack(typename E::raw* row, const Pack<E, V>& p, int c, int H) {
  if constexpr (VEC) {
    store_pack<E, V>(row + c, p);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(&p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if (c + V <= H) store_inner<(int)sizeof(typename E::raw)>(row + c, w);
    else store_any<(int)sizeof(typename E::raw)>(row + c, w, H - c);
  }
}
// The pack's weights; single loads where they are not aligned or the row ends
// inside the pack.
template <typename E, bool WF32, int V, bool VEC>
__device__ __forceinline__ void row_weights(float (&o)[V], const void* w, int c, int H, float def) {
  if (VEC || (((uintptr_t)w & 15) == 0 && c + V <= H)) {
    weights_at<E, WF32, V>(o, w, c, def);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = c + j < H ? weight_at<E, WF32>(w, c + j, def) : 0.f;
  }
}

// Rows per CTA: 1 with BLOCK, else one per warp.
template <typename E, bool WF32, int NV, bool BLOCK, bool VEC>
__global__ void __launch_bounds__(BLOCK ? kNormMaxThreads : kWarpRowThreads) k_norm_fwd(NormArgs a) {
  using raw = typename E::raw;
  constexpr int V = 16 / (int)sizeof(raw);
  pdl_enter();
  __shared__ float2 red[2][kNormMaxThreads / 32];
  const int tpr = BLOCK ? blockDim.x : 32, t = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int nw = tpr / 32, rpb = BLOCK ? 1 : blockDim.x / 32;
  const float inv_h = 1.0f / (float)a.H;
  for (int64_t row = (int64_t)blockIdx.x * rpb + (BLOCK ? 0 : threadIdx.x / 32); row < a.T;
       row += (int64_t)gridDim.x * rpb) {
    const raw* x = reinterpret_cast<const raw*>(a.x) + row * a.ldx;
    Pack<E, V> p[NV];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < a.H) load_row_pack<E, V, VEC>(p[i], x, c, a.H);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * tpr + t) * V < a.H) {
#pragma unroll
        for (int j = 0; j < V; ++j) s += E::to(p[i].v[j]);
      }
    const float mu = row_sum<BLOCK>(s, red[0], nw) * inv_h;
    float m2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * tpr + t) * V < a.H) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!VEC && (i * tpr + t) * V + j >= a.H) continue;
          const float d = E::to(p[i].v[j]) - mu;
          m2 = fmaf(d, d, m2);
        }
      }
    const float r = rsqrtf(row_sum<BLOCK>(m2, red[1], nw) * inv_h + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
    raw* y = reinterpret_cast<raw*>(a.out) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < a.H) {
        float g[V], b[V];
        row_weights<E, WF32, V, VEC>(g, a.gamma, c, a.H, 1.f);
        row_weights<E, WF32, V, VEC>(b, a.beta, c, a.H, 0.f);
        Pack<E, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = E::from(fmaf((E::to(p[i].v[j]) - mu) * r, g[j], b[j]));
        store_row_pack<E, V, VEC>(y, o, c, a.H);
      }
    }
  }
}

// Rows too long for the registers of one CTA: the row is read three times
// (the later reads come from L2).
template <typename E, bool WF32>
__global__ void __launch_bounds__(kNormMaxThreads) k_norm_fwd_long(NormArgs a) {
  using raw = typename E::raw;
  pdl_enter();
  __shared__ float2 red[2][kNormMaxThreads / 32];
  const int nw = blockDim.x / 32;
  const float inv_h = 1.0f / (float)a.H;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const raw* x = reinterpret_cast<const raw*>(a.x) + row * a.ldx;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) s += E::to(x[c]);
    const float mu = row_sum<true>(s, red[0], nw) * inv_h;
    float m2 = 0.f;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float d = E::to(x[c]) - mu;
      m2 = fmaf(d, d, m2);
    }
    const float r = rsqrtf(row_sum<true>(m2, red[1], nw) * inv_h + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
    raw* y = reinterpret_cast<raw*>(a.out) + row * a.ldo;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x)
      y[c] = E::from(fmaf((E::to(x[c]) - mu) * r, weight_at<E, WF32>(a.gamma, c, 1.f),
                          weight_at<E, WF32>(a.beta, c, 0.f)));
  }
}

// PART: the weight's gradient is wanted. Partial row p = the CTA:
// part[p][0][c] = dgamma, part[p][1][c] = dbeta over its rows (of its warps,
// where they hold a row each, added in warp order).
template <typename E, bool WF32, int NV, bool BLOCK, bool PART, bool VEC>
__global__ void __launch_bounds__(BLOCK ? kNormBwdThreads : kWarpRowThreads) k_norm_bwd(NormArgs a) {
  using raw = typename E::raw;
  constexpr int V = 16 / (int)sizeof(raw);
  pdl_enter();
  __shared__ float2 red[2][kNormMaxThreads / 32];
  const int tpr = BLOCK ? blockDim.x : 32, t = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int nw = tpr / 32, rpb = BLOCK ? 1 : blockDim.x / 32;
  const int64_t slot = (int64_t)blockIdx.x * rpb + (BLOCK ? 0 : threadIdx.x / 32);
  const float inv_h = 1.0f / (float)a.H;
  float dg[PART ? NV * V : 1], db[PART ? NV * V : 1];
  if constexpr (PART) {
#pragma unroll
    for (int i = 0; i < NV * V; ++i) dg[i] = db[i] = 0.f;
  }
  int flip = 0;
  for (int64_t row = slot; row < a.T; row += (int64_t)gridDim.x * rpb, flip ^= 1) {
    const raw* x = reinterpret_cast<const raw*>(a.x) + row * a.ldx;
    const raw* dy = reinterpret_cast<const raw*>(a.dy) + row * a.lddy;
    Pack<E, V> px[NV], pd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < a.H) {
        load_row_pack<E, V, VEC>(px[i], x, c, a.H);
        load_row_pack<E, V, VEC>(pd[i], dy, c, a.H);      // zeros past the row's end: they add nothing
      }
    }
    const float mu = a.mean[row], r = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < a.H) {
        float g[V];
        row_weights<E, WF32, V, VEC>(g, a.gamma, c, a.H, 1.f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = E::to(pd[i].v[j]), xh = (E::to(px[i].v[j]) - mu) * r, tg = d * g[j];
          s1 += tg;
          s2 = fmaf(tg, xh, s2);
          if constexpr (PART) {
            dg[i * V + j] = fmaf(d, xh, dg[i * V + j]);
            db[i * V + j] += d;
          }
        }
      }
    }
    const float2 m = row_sum2<BLOCK>(s1, s2, red[flip], nw);
    const float m1 = m.x * inv_h, m2 = m.y * inv_h;
    raw* dx = reinterpret_cast<raw*>(a.out) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < a.H) {
        float g[V];
        row_weights<E, WF32, V, VEC>(g, a.gamma, c, a.H, 1.f);
        Pack<E, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (E::to(px[i].v[j]) - mu) * r;
          o.v[j] = E::from(r * (E::to(pd[i].v[j]) * g[j] - m1 - xh * m2));
        }
        store_row_pack<E, V, VEC>(dx, o, c, a.H);
      }
    }
  }
  if constexpr (PART) {
    float* pg = a.part + (int64_t)blockIdx.x * 2 * a.H;
    if constexpr (BLOCK) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * V;
        if (c < a.H) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (!VEC && c + j >= a.H) continue;
            pg[c + j] = dg[i * V + j];
            pg[a.H + c + j] = db[i * V + j];
          }
        }
      }
    } else {
      __shared__ float sums[kWarpRowThreads / 32][2][32 * V];
      const int w = threadIdx.x >> 5;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sums[w][0][t * V + j] = dg[j];
        sums[w][1][t * V + j] = db[j];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * a.H; c += kWarpRowThreads) {
        const int k = c >= a.H;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kWarpRowThreads / 32; ++i) v += sums[i][k][c - k * a.H];
        pg[c] = v;
      }
    }
  }
}

// ---- many rows: a ring of rows in shared memory ---------------------------------
// Registers alone keep too few bytes in flight (a row's barriers come between
// its loads and the next row's): thread 0 keeps kRing bulk copies of rows
// ahead in shared memory. A stage is refilled behind the row's first barrier,
// when every thread has its packs in registers.
constexpr int kRingMax = 8;
constexpr int kRingBytes = 200 * 1024;    // of an SM's shared memory, for all its CTAs
constexpr int kRingHead = 128;            // barriers, in front of the stages

// The bounded wait for a row. A copy from this GPU's memory always lands;
// should the wait run out all the same, the row's results become NaN, and the
// thread's columns of the weight's gradient with them.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity) {
  volatile int give_up = 0;
  return tc::mbar_wait(bar, parity, &give_up);
}

// Bytes of a row of `bytes` from p as a stage holds them: from the 16-byte
// boundary at or before p, with a unit to spare behind.
__host__ __device__ inline uint32_t ring_row_bytes(uint32_t bytes, bool any) {
  return any ? (bytes + 15) / 16 * 16 + 32 : bytes;
}
// ANY: a row at any alignment, copied with the rest of the 16-byte units that
// it starts and ends in. Those belong to the rows before and after it; the
// first row's head and the last row's tail, where there may be nothing, go
// element by element.
template <typename raw, bool ANY>
__device__ __forceinline__ void ring_copy(uint8_t* d, const raw* p, uint32_t bytes, bool head, bool tail, uint64_t* bar) {
  if constexpr (!ANY) {
    tc::mbar_arrive_expect_tx(bar, bytes);
    tc::bulk_g2s_plain(d, p, bytes, bar);
  } else {
    const uint8_t* lo = reinterpret_cast<const uint8_t*>(p);
    const uint8_t* hi = lo + bytes;
    const uint8_t* a = reinterpret_cast<const uint8_t*>((uintptr_t)lo & ~(uintptr_t)15);
    const uint8_t* b = reinterpret_cast<const uint8_t*>(((uintptr_t)hi + 15) & ~(uintptr_t)15);
    const uint8_t* base = a;
    if (head && a != lo) {
      a += 16;
      for (const uint8_t* e = lo; e < a && e < hi; e += sizeof(raw))
        *reinterpret_cast<raw*>(d + (e - base)) = *reinterpret_cast<const raw*>(e);
    }
    if (tail && b != hi) {
      b -= 16;
      for (const uint8_t* e = b < lo ? lo : b; e < hi; e += sizeof(raw))
        *reinterpret_cast<raw*>(d + (e - base)) = *reinterpret_cast<const raw*>(e);
    }
    const uint32_t n = b > a ? (uint32_t)(b - a) : 0u;
    tc::mbar_arrive_expect_tx(bar, n);
    if (n) tc::bulk_g2s_plain(d + (a - base), a, n, bar);
  }
}

template <typename E, bool WF32, int NV, bool PART, bool BWD, bool ANY>
__global__ void __launch_bounds__(kNormBwdThreads) k_norm_ring(NormArgs a, int stages) {
  using raw = typename E::raw;
  constexpr int V = 16 / (int)sizeof(raw), NP = V / 2;      // pairs of a pack
  pdl_enter();
  __shared__ float4 red[2][kNormBwdThreads / 32];
  extern __shared__ __align__(128) uint8_t ring[];
  uint64_t* full = reinterpret_cast<uint64_t*>(ring);
  const uint32_t bytes = (uint32_t)a.H * sizeof(raw), row_bytes = ring_row_bytes(bytes, ANY);
  const uint32_t stage_bytes = row_bytes * (BWD ? 2 : 1);
  const int tpr = blockDim.x, t = threadIdx.x, nw = tpr / 32;
  const float inv_h = 1.0f / (float)a.H;
  const raw* X = reinterpret_cast<const raw*>(a.x);
  const raw* DY = reinterpret_cast<const raw*>(a.dy);
  auto fetch = [&](int s, int64_t row) {
    if (row >= a.T) return;
    uint8_t* d = ring + kRingHead + s * stage_bytes;
    ring_copy<raw, ANY>(d, X + row * a.ldx, bytes, row == 0, row == a.T - 1, &full[s]);
    if (BWD) ring_copy<raw, ANY>(d + row_bytes, DY + row * a.lddy, bytes, row == 0, row == a.T - 1, &full[s]);
  };
  // pack c of the row in a stage; ANY: elements past the row's end are zeros
  auto pack_of = [&](Pack<E, V>& p, const uint8_t* src, const raw* row, int c) {
    if constexpr (!ANY) {
      load_pack(p, reinterpret_cast<const raw*>(src) + c * V);
    } else {
      const int off = (int)((uintptr_t)row & 15);
      const uint4 u0 = reinterpret_cast<const uint4*>(src)[c], u1 = reinterpret_cast<const uint4*>(src)[c + 1];
      uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w}, r4[4];
      shift_units<(int)sizeof(raw), 16>(r4, w, off);
      *reinterpret_cast<uint4*>(&p) = make_uint4(r4[0], r4[1], r4[2], r4[3]);
      if (c * V + V > a.H) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c * V + j >= a.H) p.v[j] = 0;
      }
    }
  };
  if (t == 0) {
    for (int s = 0; s < stages; ++s) tc::mbar_init(&full[s], BWD ? 2 : 1);
    tc::fence_mbar_init();
    for (int s = 0; s < stages; ++s) fetch(s, blockIdx.x + (int64_t)s * gridDim.x);
  }
  __syncthreads();
  // the thread's columns are the same in every row: weights stay in registers
  f32x2 g[NV][NP], b[BWD ? 1 : NV][NP];
  f32x2 dg[PART ? NV : 1][NP], db[PART ? NV : 1][NP];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + t) * V;
    float w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = 0.f;
    if (c < a.H) row_weights<E, WF32, V, !ANY>(w, a.gamma, c, a.H, 1.f);
#pragma unroll
    for (int j = 0; j < NP; ++j) g[i][j] = pack2(w[2 * j], w[2 * j + 1]);
    if constexpr (!BWD) {
      if (c < a.H) row_weights<E, WF32, V, !ANY>(w, a.beta, c, a.H, 0.f);
#pragma unroll
      for (int j = 0; j < NP; ++j) b[i][j] = pack2(w[2 * j], w[2 * j + 1]);
    }
    if constexpr (PART) {
#pragma unroll
      for (int j = 0; j < NP; ++j) dg[i][j] = db[i][j] = 0;
    }
  }
  // One pack a thread: two rows go round together, which halves the barriers a
  // row waits for and shares their shuffles (at 16384 x 2880 forward 51 -> 47
  // us, backward 75 -> 65). Not in the backward at odd alignments, where the
  // shifted loads take the registers (101 against 125 us at 16384 x 2881).
  constexpr int RW = NV == 1 && !(BWD && ANY) ? 2 : 1;
  const int64_t step = gridDim.x;
  float mu[RW], r[RW], mu_next[RW], r_next[RW];
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    mu[k] = r[k] = mu_next[k] = r_next[k] = 0.f;
    const int64_t row = blockIdx.x + k * step;
    if (BWD && row < a.T) {
      mu_next[k] = a.mean[row];
      r_next[k] = a.rstd[row];
    }
  }
  int s = 0;
  uint32_t parity = 0;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += RW * step) {
    const bool two = RW == 2 && row + step < a.T;
    Pack<E, V> px[RW][NV], pd[RW][BWD ? NV : 1];
    float bad[RW];
    int stage[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const int64_t rk = row + k * step;
      if (BWD) {
        mu[k] = mu_next[k];
        r[k] = r_next[k];
        if (rk + RW * step < a.T) {
          mu_next[k] = a.mean[rk + RW * step];
          r_next[k] = a.rstd[rk + RW * step];
        }
      }
      stage[k] = s;
      bad[k] = 0.f;
      if (k == 0 || two) {
        bad[k] = ring_wait(&full[s], parity) ? 0.f : __int_as_float(0x7fffffff);
        const uint8_t* sx = ring + kRingHead + s * stage_bytes;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = i * tpr + t;
          if (c * V < a.H) {
            pack_of(px[k][i], sx, X + rk * a.ldx, c);
            if constexpr (BWD) pack_of(pd[k][i], sx + row_bytes, DY + rk * a.lddy, c);
          }
        }
        if (++s == stages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    // behind the first barrier: every thread has its packs, the stages are free
    auto refill = [&]() {
      if (t == 0) {
#pragma unroll
        for (int k = 0; k < RW; ++k)
          if (k == 0 || two) fetch(stage[k], row + (k + (int64_t)stages) * step);
      }
    };
    if constexpr (BWD) {
      // one pack a thread: xh and dy gamma are kept for the second pass
      constexpr bool kKeep = NV == 1;
      f32x2 xk[RW][kKeep ? NP : 1], tk[RW][kKeep ? NP : 1];
      float s1[RW], s2[RW];
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const f32x2 nmu = pack2(-mu[k], -mu[k]), rr = pack2(r[k], r[k]);
        f32x2 p1 = pack2(PART ? 0.f : bad[k], 0.f), p2 = 0;
        if (PART && bad[k] != 0.f) {      // a NaN dy reaches the row's sums and the columns'
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) pd[k][i].v[j] = E::from(bad[k]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((k == 0 || two) && (i * tpr + t) * V < a.H) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const f32x2 d = pd[k][i].pair(j), xh = mul2(add2(px[k][i].pair(j), nmu), rr), tg = mul2(d, g[i][j]);
              p1 = add2(p1, tg);
              p2 = fma2(tg, xh, p2);
              if constexpr (kKeep) {
                xk[k][j] = xh;
                tk[k][j] = tg;
              }
              if constexpr (PART) {
                dg[i][j] = fma2(d, xh, dg[i][j]);
                db[i][j] = add2(db[i][j], d);
              }
            }
          }
        const float2 u1 = unpack2(p1), u2 = unpack2(p2);
        s1[k] = u1.x + u1.y;
        s2[k] = u2.x + u2.y;
      }
      if constexpr (RW == 2) {
        const float4 m = row_sum4(s1[0], s2[0], s1[1], s2[1], red[flip], nw);
        s1[0] = m.x; s2[0] = m.y; s1[1] = m.z; s2[1] = m.w;
      } else {
        const float2 m = row_sum2<true>(s1[0], s2[0], reinterpret_cast<float2*>(red[flip]), nw);
        s1[0] = m.x; s2[0] = m.y;
      }
      flip ^= 1;
      refill();
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        if (k == 1 && !two) break;
        raw* out = reinterpret_cast<raw*>(a.out) + (row + k * step) * a.ldo;
        // r (t - m1 - xh m2)
        const float m1 = -r[k] * (s1[k] * inv_h), m2 = -r[k] * (s2[k] * inv_h);
        const f32x2 nmu = pack2(-mu[k], -mu[k]), rr = pack2(r[k], r[k]), nm1 = pack2(m1, m1), nm2 = pack2(m2, m2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * tpr + t) * V;
          if (c < a.H) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              if constexpr (kKeep) {
                o.set_pair(j, fma2(tk[k][j], rr, fma2(xk[k][j], nm2, nm1)));
              } else {
                const f32x2 xh = mul2(add2(px[k][i].pair(j), nmu), rr);
                o.set_pair(j, fma2(mul2(pd[k][i].pair(j), g[i][j]), rr, fma2(xh, nm2, nm1)));
              }
            }
            store_row_pack<E, V, !ANY>(out, o, c, a.H);
          }
        }
      }
    } else {
      float sum[RW], m2[RW];
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        f32x2 p = pack2(bad[k], 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((k == 0 || two) && (i * tpr + t) * V < a.H) {
#pragma unroll
            for (int j = 0; j < NP; ++j) p = add2(p, px[k][i].pair(j));
          }
        const float2 u = unpack2(p);
        sum[k] = u.x + u.y;
      }
      if constexpr (RW == 2) {
        const float2 m = row_sum2<true>(sum[0], sum[1], reinterpret_cast<float2*>(red[0]), nw);
        mu[0] = m.x * inv_h;
        mu[1] = m.y * inv_h;
      } else {
        mu[0] = row_sum<true>(sum[0], reinterpret_cast<float2*>(red[0]), nw) * inv_h;
      }
      refill();
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const f32x2 nmu = pack2(-mu[k], -mu[k]);
        f32x2 p = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((k == 0 || two) && (i * tpr + t) * V < a.H) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              f32x2 d = add2(px[k][i].pair(j), nmu);
              if (ANY) {                                  // past the row's end
                const int c = (i * tpr + t) * V + 2 * j;
                if (c + 1 >= a.H) d = c >= a.H ? 0 : pack2(unpack2(d).x, 0.f);
              }
              p = fma2(d, d, p);
            }
          }
        const float2 u = unpack2(p);
        m2[k] = u.x + u.y;
      }
      if constexpr (RW == 2) {
        const float2 m = row_sum2<true>(m2[0], m2[1], reinterpret_cast<float2*>(red[1]), nw);
        r[0] = rsqrtf(m.x * inv_h + a.eps);
        r[1] = rsqrtf(m.y * inv_h + a.eps);
      } else {
        r[0] = rsqrtf(row_sum<true>(m2[0], reinterpret_cast<float2*>(red[1]), nw) * inv_h + a.eps);
      }
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        if (k == 1 && !two) break;
        const int64_t rk = row + k * step;
        if (t == 0) {
          if (a.mean) a.mean[rk] = mu[k];
          if (a.rstd) a.rstd[rk] = r[k];
        }
        raw* out = reinterpret_cast<raw*>(a.out) + rk * a.ldo;
        const f32x2 nmu = pack2(-mu[k], -mu[k]), rr = pack2(r[k], r[k]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * tpr + t) * V;
          if (c < a.H) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < NP; ++j)
              o.set_pair(j, fma2(mul2(add2(px[k][i].pair(j), nmu), rr), g[i][j], b[i][j]));
            store_row_pack<E, V, !ANY>(out, o, c, a.H);
          }
        }
      }
    }
  }
  if constexpr (PART) {
    float* pg = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < a.H) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float2 u = unpack2(dg[i][j]), v = unpack2(db[i][j]);
          if (!ANY || c + 2 * j < a.H) {
            pg[c + 2 * j] = u.x;
            pg[a.H + c + 2 * j] = v.x;
          }
          if (!ANY || c + 2 * j + 1 < a.H) {
            pg[c + 2 * j + 1] = u.y;
            pg[a.H + c + 2 * j + 1] = v.y;
          }
        }
      }
    }
  }
}

// dx of rows too long for registers (three reads), without the weight's
// gradient.
template <typename E, bool WF32>
__global__ void __launch_bounds__(kNormMaxThreads) k_norm_bwd_long(NormArgs a) {
  using raw = typename E::raw;
  pdl_enter();
  __shared__ float2 red[2][kNormMaxThreads / 32];
  const int nw = blockDim.x / 32;
  const float inv_h = 1.0f / (float)a.H;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
    const raw* x = reinterpret_cast<const raw*>(a.x) + row * a.ldx;
    const raw* dy = reinterpret_cast<const raw*>(a.dy) + row * a.lddy;
    const float mu = a.mean[row], r = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float tg = E::to(dy[c]) * weight_at<E, WF32>(a.gamma, c, 1.f);
      s1 += tg;
      s2 = fmaf(tg, (E::to(x[c]) - mu) * r, s2);
    }
    const float2 m = row_sum2<true>(s1, s2, red[flip], nw);
    const float m1 = m.x * inv_h, m2 = m.y * inv_h;
    raw* dx = reinterpret_cast<raw*>(a.out) + row * a.ldo;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float tg = E::to(dy[c]) * weight_at<E, WF32>(a.gamma, c, 1.f);
      dx[c] = E::from(r * (tg - m1 - (E::to(x[c]) - mu) * r * m2));
    }
  }
}

// Partial rows of the weight's gradient of long rows: thread = column, block
// row p takes rows p, p + P, ...
template <typename E>
__global__ void __launch_bounds__(256) k_norm_dw_long(NormArgs a) {
  using raw = typename E::raw;
  pdl_enter();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float dg = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const float d = E::to(reinterpret_cast<const raw*>(a.dy)[row * a.lddy + c]);
    dg = fmaf(d, (E::to(reinterpret_cast<const raw*>(a.x)[row * a.ldx + c]) - a.mean[row]) * a.rstd[row], dg);
    db += d;
  }
  float* p = a.part + (int64_t)blockIdx.y * 2 * a.H;
  p[c] = dg;
  p[a.H + c] = db;
}

// dgamma / dbeta = the P partial rows added in a fixed order: 32 columns a
// block, row lane l adds partial rows l, l + 32, ..., then the lanes in order.
template <typename E, bool WF32>
__global__ void __launch_bounds__(1024) k_norm_dw_sum(const float* __restrict__ part, int P, int H, void* dgamma,
                                                      void* dbeta) {
  pdl_enter();
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), l = threadIdx.x >> 5;
  const int64_t at = (int64_t)blockIdx.y * H + c;
  float v = 0.f;
  if (c < H) {
    for (int p = l; p < P; p += 10 * 32) {      // ten loads in flight
      float t[10];
#pragma unroll
      for (int j = 0; j < 10; ++j) t[j] = p + 32 * j < P ? part[(int64_t)(p + 32 * j) * 2 * H + at] : 0.f;
#pragma unroll
      for (int j = 0; j < 10; ++j) v += t[j];
    }
  }
  s[l][threadIdx.x & 31] = v;
  __syncthreads();
  if (l == 0 && c < H) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    void* d = blockIdx.y == 0 ? dgamma : dbeta;
    if (d) {
      if constexpr (WF32) reinterpret_cast<float*>(d)[c] = sum;
      else reinterpret_cast<typename E::raw*>(d)[c] = E::from(sum);
    }
  }
}

// ---- host ---------------------------------------------------------------------
static bool on(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// 16-byte accesses: every row of x, dy and out, and the weights, start on 16
// bytes and H is a whole number of packs.
static bool vec_ok(const NormArgs& a, int esize) {
  const int V = 16 / esize;
  const bool rows = a.H % V == 0 && a.ldx % V == 0 && a.ldo % V == 0 && on(a.x, 16) && on(a.out, 16) &&
                    (!a.dy || (a.lddy % V == 0 && on(a.dy, 16)));
  return rows && on(a.gamma, 16) && on(a.beta, 16);
}

struct NormPlan {
  bool longrow, block;
  int nv, threads;
  int64_t grid;
};
// Threads and packs a thread for rows of n packs. resident: threads an SM
// holds, for a grid that is resident at once and whose CTAs sum over rows (at
// most max_parts of them where that is not 0); 0: a CTA a row, handed out as
// SMs come free.
static NormPlan norm_plan(int64_t n, int64_t T, int resident, int max_parts, int max_threads) {
  NormPlan p = {};
  if (n <= 32) {                       // a warp a row
    p.nv = 1;
    p.threads = kWarpRowThreads;
  } else {
    p.block = true;
    // fewest packs a thread (one, two, four) that leave at most 256 threads a
    // row: short barriers, several rows in flight on an SM
    p.nv = 1;
    while (p.nv < 4 && (n + p.nv - 1) / p.nv > 256) p.nv *= 2;
    p.threads = (int)(((n + p.nv - 1) / p.nv + 31) / 32 * 32);
    if (p.threads > max_threads) p.longrow = true;
  }
  if (p.longrow) p.threads = kNormMaxThreads;
  const int rpb = p.block ? 1 : p.threads / 32;
  int64_t g = p.block && !resident ? INT32_MAX
                                   : (int64_t)device_sms() * std::max(1, (resident ? resident : 2048) / p.threads);
  if (max_parts) g = std::min<int64_t>(g, max_parts);
  p.grid = std::max<int64_t>(1, std::min<int64_t>(g, (T + rpb - 1) / rpb));
  return p;
}

// Launch of the ring, or cudaErrorNotSupported: few rows, rows of at most a
// warp's packs (many rows in flight already) or of more than the registers hold.
template <typename E, bool WF32, int NV, bool PART, bool BWD, bool ANY>
static cudaError_t ring_nv(const NormArgs& a, int threads, int64_t* parts, cudaStream_t st) {
  const auto kern = k_norm_ring<E, WF32, NV, PART, BWD, ANY>;
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    regs.store((at.numRegs + 7) / 8 * 8, std::memory_order_release);
  }
  static std::atomic<bool> done[kMaxDevices] = {};
  cudaError_t e = set_smem_once((const void*)kern, kRingBytes + 1024, done);
  if (e != cudaSuccess) return e;
  const int stage = (int)ring_row_bytes((uint32_t)a.H * sizeof(typename E::raw), ANY) * (BWD ? 2 : 1);
  // CTAs an SM holds (registers are handed out to four warps at a time), each
  // with at least two stages; then all the stages that fit
  int ctas = std::max(1, std::min({6, 65536 / (regs.load() * ((threads + 127) / 128 * 128)), 2048 / threads}));
  while (ctas > 1 && 2 * stage * ctas > kRingBytes) --ctas;
  const int stages = std::min(kRingMax, kRingBytes / (ctas * stage));
  if (stages < 2) return cudaErrorNotSupported;
  const int64_t grid = std::min<int64_t>({a.T, (int64_t)device_sms() * ctas, kNormMaxParts});
  *parts = grid;
  note_launch();
  return launch_pdl(kern, dim3((unsigned)grid), dim3(threads), (size_t)kRingHead + (size_t)stages * stage, st, a, stages);
}
template <typename E, bool WF32, bool PART, bool BWD, bool ANY>
static cudaError_t ring_launch(const NormArgs& a, int64_t* parts, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(typename E::raw);
  const int n = (a.H + V - 1) / V;
  // The backward's two inputs, in a CTA's registers, leave few bytes in flight:
  // 16384 x 2880 65.6 us against 97.8 with rows in registers, 300 x 2880 10.1
  // against 13.8, 32 x 2880 8.4 and 8.3.
  if (n <= 32 || n > 4 * kNormBwdThreads || 2 * a.T < (BWD ? device_sms() : 0)) return cudaErrorNotSupported;
  // one pack a thread while that is at most 512 threads, then two, four: the
  // sums over rows of a thread's columns stay in registers, and the fewer of
  // them the more warps hide the row's barriers
  const int nv = n <= kNormBwdThreads ? 1 : n <= 2 * kNormBwdThreads ? 2 : 4;
  const int threads = ((n + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1) return ring_nv<E, WF32, 1, PART, BWD, ANY>(a, threads, parts, st);
  return nv == 2 ? ring_nv<E, WF32, 2, PART, BWD, ANY>(a, threads, parts, st)
                 : ring_nv<E, WF32, 4, PART, BWD, ANY>(a, threads, parts, st);
}

template <typename E, bool WF32, bool VEC>
static cudaError_t fwd_v(const NormArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(typename E::raw);
  // The ring gains only in many long rows of 16 bits (16384 x 2880 47.2 us, 49.9
  // with rows in registers; 9000 x 2880 27.6 and 28.6; but 4096 x 2880 13.8 and
  // 12.9, 16384 x 1000 23.6 and 20.8), which at odd alignments it slows down
  // (16384 x 2881 84 and 77), and in fp32 at odd alignments (8192 x 2881 44.9 and
  // 59.1, 1000 x 2881 8.2 and 9.7; aligned, 16384 x 2880, 69 and 59).
  constexpr bool k32 = sizeof(typename E::raw) == 4;
  if constexpr (k32 != VEC) {
    int64_t parts;
    if (a.T >= (k32 ? 4LL : 48LL) * device_sms() && (k32 || a.H > 256 * V)) {
      const cudaError_t re = ring_launch<E, WF32, false, false, !VEC>(a, &parts, st);
      if (re != cudaErrorNotSupported) return re;
    }
  }
  const NormPlan p = norm_plan(((int64_t)a.H + V - 1) / V, a.T, 0, 0, kNormMaxThreads);
  const dim3 g((unsigned)p.grid), b(p.threads);
  note_launch();
  if (p.longrow) return launch_pdl(k_norm_fwd_long<E, WF32>, g, b, 0, st, a);
  if (!p.block) return launch_pdl(k_norm_fwd<E, WF32, 1, false, VEC>, g, b, 0, st, a);
  if (p.nv == 1) return launch_pdl(k_norm_fwd<E, WF32, 1, true, VEC>, g, b, 0, st, a);
  if (p.nv == 2) return launch_pdl(k_norm_fwd<E, WF32, 2, true, VEC>, g, b, 0, st, a);
  return launch_pdl(k_norm_fwd<E, WF32, 4, true, VEC>, g, b, 0, st, a);
}

template <typename E, bool WF32, int NV, bool BLOCK, bool VEC>
static cudaError_t bwd_launch(const NormArgs& a, const NormPlan& p, cudaStream_t st) {
  const dim3 g((unsigned)p.grid), b(p.threads);
  note_launch();
  if (a.dgamma || a.dbeta) return launch_pdl(k_norm_bwd<E, WF32, NV, BLOCK, true, VEC>, g, b, 0, st, a);
  return launch_pdl(k_norm_bwd<E, WF32, NV, BLOCK, false, VEC>, g, b, 0, st, a);
}

template <typename E, bool WF32, bool VEC>
static cudaError_t bwd_v(const NormArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(typename E::raw);
  const bool want = a.dgamma || a.dbeta;
  const NormPlan p = norm_plan(((int64_t)a.H + V - 1) / V, a.T, (int64_t)a.H <= 32 * V ? 2048 : 512,
                               want ? kNormMaxParts : 0, kNormBwdThreads);
  cudaError_t e = cudaErrorNotSupported;
  int64_t parts = p.grid;
  e = want ? ring_launch<E, WF32, true, true, !VEC>(a, &parts, st) : ring_launch<E, WF32, false, true, !VEC>(a, &parts, st);
  if (e != cudaErrorNotSupported) {
  } else if (p.longrow) {
    note_launch();
    e = launch_pdl(k_norm_bwd_long<E, WF32>, dim3((unsigned)p.grid), dim3(p.threads), 0, st, a);
    if (e != cudaSuccess) return e;
    if (want) {
      const int cb = (a.H + 255) / 256;
      parts = std::min<int64_t>(std::min<int64_t>(a.T, kNormMaxParts), std::max(1, device_sms() * 8 / cb));
      note_launch();
      e = launch_pdl(k_norm_dw_long<E>, dim3(cb, (unsigned)parts), dim3(256), 0, st, a);
    }
  } else if (!p.block) {
    e = bwd_launch<E, WF32, 1, false, VEC>(a, p, st);
  } else if (p.nv == 1) {
    e = bwd_launch<E, WF32, 1, true, VEC>(a, p, st);
  } else if (p.nv == 2) {
    e = bwd_launch<E, WF32, 2, true, VEC>(a, p, st);
  } else {
    e = bwd_launch<E, WF32, 4, true, VEC>(a, p, st);
  }
  if (e != cudaSuccess || !want) return e;
  note_launch();
  return launch_pdl(k_norm_dw_sum<E, WF32>, dim3((a.H + 31) / 32, 2), dim3(1024), 0, st, (const float*)a.part,
                    (int)parts, a.H, a.dgamma, a.dbeta);
}

template <typename E, bool WF32, bool FWD>
static cudaError_t by_vec(const NormArgs& a, cudaStream_t st) {
  const bool vec = vec_ok(a, sizeof(typename E::raw));
  if constexpr (FWD) return vec ? fwd_v<E, WF32, true>(a, st) : fwd_v<E, WF32, false>(a, st);
  else return vec ? bwd_v<E, WF32, true>(a, st) : bwd_v<E, WF32, false>(a, st);
}

template <bool FWD>
static cudaError_t by_type(const NormArgs& a, cudaStream_t st) {
  if (a.dtype == MOE_DT_F32) return by_vec<F32, true, FWD>(a, st);
  if (a.dtype == MOE_DT_F16)
    return a.wdtype == MOE_DT_F32 ? by_vec<F16, true, FWD>(a, st) : by_vec<F16, false, FWD>(a, st);
  return a.wdtype == MOE_DT_F32 ? by_vec<Bf16, true, FWD>(a, st) : by_vec<Bf16, false, FWD>(a, st);
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) { return by_type<true>(a, st); }
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) { return by_type<false>(a, st); }

}  // namespace moe
