// The routed layer for a few tokens with experts in 16 bits, in two launches:
// the router (logits, top-k, weights) here, everything behind it in few16.cu.
//
// The router's product x . W_r streams W_r [H, E] fp32 once for every eight
// tokens: the reduction is cut into slices, a CTA each, whose partial sums the last
// CTA to arrive (of those eight tokens') adds in order and routes. 1 x 7168 x 256:
// latency, not the 7.3 MB; so all of a thread's rows are asked for at once, and a small
// product is one CTA's, without a join. What the router adds to a layer with ready ids, in us,
// tokens x H x experts: one CTA's 1 x 256 x 8 2.2, 1 x 2048 x 8 3.5; joined 1 x 2880 x 128 6.3, 1 x
// 7168 x 256 8.0 to 8.7, 5 x 1999 x 24 7.6, 16 x 2880 x 24 7.5, x 128 10, 16 x 7168 x 256 14; 64 x 2880 x 128 9.8, 64
// x 7168 x 256 18.
#include "few16.cuh"

namespace moe {

static int64_t al256(int64_t v) { return (v + 255) / 256 * 256; }

constexpr int kRThreads = 512;
constexpr int kRTokens = 8;           // most tokens of a CTA
constexpr int kRChunk = 4096;         // values of x in shared memory at a time
constexpr int kRRows = 8;             // rows of W_r that a thread asks for at once
static_assert(MOE_LAYER16_MAX_T <= kRTokens * kL16Arrive, "an arrival counter for every kRTokens tokens");

struct RoutePlan {
  int tt;               // tokens a CTA
  int quads;            // of experts a CTA: a power of two up to 64
  int et, z, ks;        // expert tiles, groups of tt tokens, slices of H
  int ep;               // experts, rounded up to 4
  int64_t floats() const { return (int64_t)z * ks * tt * ep; }
};
static RoutePlan route_plan(int T, int H, int E) {
  RoutePlan p;
  p.tt = T == 1 ? 1 : T == 2 ? 2 : T <= 4 ? 4 : kRTokens;
  p.z = (T + p.tt - 1) / p.tt;
  p.ep = (E + 3) / 4 * 4;
  p.quads = 1;
  while (p.quads < 64 && p.quads * 4 < E) p.quads *= 2;
  p.et = (E + p.quads * 4 - 1) / (p.quads * 4);
  // a CTA for every SM, at least 16 rows of H each, and no more partial sums than
  // the last CTA reads in about 40 loads a thread
  const int items = p.tt * (p.ep / 4);
  p.ks = std::max(1, std::min({kFewSms / (p.z * p.et), H / 16, 40 * kRThreads / items}));
  // One CTA alone where it asks for all rows at once and needs no join: the layer of 1
  // token, 256 x 128 x 8, 15.4 us against 18.3; 1 x 2048 x 8 21.1, 24.0; 8 x 256 x 64 40.1, 41.4. Where
  // it needs more rounds, it is the slower: 8 x 1024 x 8 30.9, 28.8; 1 x 1024 x 64 no gain.
  if (p.et == 1 && H <= kRRows * (kRThreads / p.quads) && H * p.tt <= kRChunk) p.ks = 1;
  return p;
}
// Floats of partial sums that suffice for T tokens and any fewer.
static int64_t route_floats(int T, int H, int E) {
  int64_t most = 0;
  for (int t = 1, before = 0; before < T; before = t, t += std::min(t, kRTokens))      // a plan holds for a range of T
    most = std::max(most, route_plan(std::min(t, T), H, E).floats());
  return most;
}

// Workspace: the counters, y [2 parts][T (k + S)][I] 16-bit rows by group, the sums of parts
// of the groups, the router's partial sums.
constexpr int kCounters = 16 + kFewSms;
struct Layer16Ws {
  int64_t ldy, y, part, router, bytes;
};
static Layer16Ws layer16_ws(int T, int H, int I, int E, int k, int S) {
  Layer16Ws w;
  w.ldy = (I + 7) / 8 * 8;
  w.y = al256(kCounters * 4);
  w.part = w.y + al256(2 * (int64_t)T * (k + S) * w.ldy * 2);
  w.router = w.part + (int64_t)kFewSms * T * 128 * 4;
  w.bytes = w.router + al256(route_floats(T, H, E) * 4);
  return w;
}
int64_t layer16_ws_bytes(int T, int H, int I, int E, int k, int S) { return layer16_ws(T, H, I, E, k, S).bytes; }

struct RouteArgs16 {
  Layer16Args a;
  RoutePlan p;
  float* part;          // [z][ks][tt][ep]
};

// Sums of a float4 over `n` partial sums, `step` floats apart, kRAhead at a time.
constexpr int kRAhead = 20;
__device__ __forceinline__ float4 sum_parts(const float* p, int n, int64_t step) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < n; i += kRAhead) {
    float4 v[kRAhead];
#pragma unroll
    for (int j = 0; j < kRAhead; ++j)
      v[j] = i + j < n ? __ldcg(reinterpret_cast<const float4*>(p + (i + j) * step)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kRAhead; ++j) { s.x += v[j].x; s.y += v[j].y; s.z += v[j].z; s.w += v[j].w; }
  }
  return s;
}

template <typename E, int TT>
__global__ void __launch_bounds__(kRThreads) k_l16_route(const RouteArgs16 r) {
  extern __shared__ __align__(16) uint8_t rsm[];
  __shared__ float xs[kRChunk];
  constexpr int kRows = kRChunk / TT;
  __shared__ int last;
  const Layer16Args& a = r.a;
  const RoutePlan& p = r.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_enter();
  // the products' counters, which the kernel behind this one starts from
  int32_t* counters = reinterpret_cast<int32_t*>(a.ws);
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    if (tid < kCounters) counters[tid] = 0;
  if (!a.W_r && !a.logits) return;
  const int t0 = blockIdx.z * TT, nt = min(TT, a.T - t0);
  const int64_t set = (int64_t)TT * p.ep;
  float* part = r.part + blockIdx.z * p.ks * set;
  const bool alone = a.W_r && p.ks * p.et == 1;
  uint32_t* keys = reinterpret_cast<uint32_t*>(rsm);          // [nt][ep] of the logits
  const int q4 = p.ep / 4;
  bool nan_seen = false;
  auto key = [&](float v) {
    nan_seen |= v != v;
    return logit_key(v != v ? -INFINITY : v);
  };

  if (a.W_r) {
    // ---- a slice of the product ----
    const int tq = tid & (p.quads - 1), rows = kRThreads / p.quads, tr = tid / p.quads;
    const int e0 = (blockIdx.y * p.quads + tq) * 4;
    const int h0 = (int)((int64_t)a.H * blockIdx.x / p.ks), h1 = (int)((int64_t)a.H * (blockIdx.x + 1) / p.ks);
    const bool vec = a.E % 4 == 0 && ((uintptr_t)a.W_r & 15) == 0;
    float acc[TT][4] = {};
    for (int hb = h0; hb < h1; hb += kRows) {
      const int n = min(kRows, h1 - hb);
      __syncthreads();
      for (int i = tid; i < n * TT; i += kRThreads) {
        const int t = i / n, h = i - t * n;
        xs[h * TT + t] = t < nt ? E::to(reinterpret_cast<const uint16_t*>(a.x)[(t0 + t) * a.ldx + hb + h]) : 0.f;
      }
      __syncthreads();
      for (int h = tr; h < n; h += rows * kRRows) {
        float w[kRRows][4];
#pragma unroll
        for (int i = 0; i < kRRows; ++i) {
          const int hh = h + i * rows;
          const float* src = a.W_r + (int64_t)(hb + hh) * a.E + e0;
          if (vec) {
            const float4 v = hh < n && e0 < a.E ? __ldg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = hh < n && e0 + j < a.E ? __ldg(src + j) : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < kRRows; ++i) {
          const int hh = h + i * rows;
          if (hh >= n) break;
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const float xv = xs[hh * TT + t];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(xv, w[i][j], acc[t][j]);
          }
        }
      }
    }
    // row lanes of a warp, then the rest through shared memory
    for (int o = p.quads; o < 32; o <<= 1)
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] += __shfl_xor_sync(kFull, acc[t][j], o);
    float* red = reinterpret_cast<float*>(rsm);               // [lanes][TT][4 quads]
    const int width = 4 * p.quads, lanes = p.quads == 64 ? 8 : 16, my = p.quads == 64 ? tr : warp;
    if (p.quads >= 32 || lane < p.quads)
#pragma unroll
      for (int t = 0; t < TT; ++t)
        *reinterpret_cast<float4*>(red + (my * TT + t) * width + 4 * tq) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    constexpr int kOwn = (TT * 256 + kRThreads - 1) / kRThreads;
    float own[kOwn];                                          // a thread's sums
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int o = tid + i * kRThreads;
      own[i] = 0.f;
      if (o >= TT * width) break;
      const int t = o / width, e = blockIdx.y * width + o - t * width;
      float v = red[o];
      for (int l = 1; l < lanes; ++l) v += red[l * TT * width + o];
      own[i] = v;
      if (!alone && e < p.ep) part[blockIdx.x * set + (int64_t)t * p.ep + e] = v;
    }
    if (alone) {
      __syncthreads();                                        // the keys lie where the sums' parts did
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int o = tid + i * kRThreads;
        if (o >= TT * width) break;
        const int t = o / width, e = o - t * width;
        if (t < nt && e < p.ep) keys[t * p.ep + e] = e < a.E ? key(own[i]) : 0u;
      }
    } else {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int old = atom_add_acq_rel_gpu(&a.arrive[blockIdx.z], 1);
        last = old == p.ks * p.et - 1;
        if (last) a.arrive[blockIdx.z] = 0;
      }
      __syncthreads();
      if (!last) return;
      __threadfence();
    }
  }

  // ---- the only or last CTA: keys of the logits, then a warp a token ----
  if (a.W_r && !alone) {
    const int items = nt * q4;
    int split = 1;                                            // threads an item
    while (2 * split * items <= kRThreads && 2 * split <= p.ks) split *= 2;
    float4* red = reinterpret_cast<float4*>(rsm + (int64_t)TT * p.ep * 4);
    for (int i = tid; i < items * split; i += kRThreads) {
      const int it = i % items, g = i / items, k0 = p.ks * g / split, k1 = p.ks * (g + 1) / split;
      red[i] = sum_parts(part + k0 * set + 4 * (int64_t)it, k1 - k0, set);
    }
    __syncthreads();
    for (int it = tid; it < items; it += kRThreads) {
      float4 v = red[it];
      for (int g = 1; g < split; ++g) {
        const float4 u = red[g * items + it];
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      const int e = it % q4 * 4;
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) keys[4 * it + j] = e + j < a.E ? key(f[j]) : 0u;
    }
  } else if (!a.W_r) {
    for (int i = tid; i < nt * p.ep; i += kRThreads) {
      const int t = i / p.ep, e = i - t * p.ep;
      keys[i] = e < a.E ? key(a.logits[(int64_t)(t0 + t) * a.E + e]) : 0u;
    }
  }
  if (nan_seen) set_status(a.status, MOE_DEV_NAN_LOGIT);
  __syncthreads();
  for (int t = warp; t < nt; t += kRThreads / 32) {
    uint32_t* row = keys + t * p.ep;
    float sel = 0.f;
    int id = 0;
    for (int j = 0; j < a.k; ++j) {
      // a lane's ids grow, so among equal keys it keeps the lowest; 0 is a taken one
      uint32_t best = 0;
      int at = 0x7fffffff;
      for (int e = lane; e < a.E; e += 32) {
        const uint32_t v = row[e];
        if (v > best) { best = v; at = e; }
      }
      const uint32_t top = __reduce_max_sync(kFull, best);
      const int win = (int)__reduce_min_sync(kFull, best == top ? (uint32_t)at : 0xffffffffu);
      if ((win & 31) == lane) row[win] = 0;
      __syncwarp();
      if (lane == j) { sel = key_logit(top); id = win; }
    }
    // softmax over the selected logits, the first of them the largest
    const float m = __shfl_sync(kFull, sel, 0);
    const float w = lane < a.k && m != -INFINITY ? expf(sel - m) : 0.f;
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) sum += __shfl_sync(kFull, w, j);
    if (lane < a.k) {
      a.ids[(t0 + t) * a.k + lane] = id;
      a.w[(t0 + t) * a.k + lane] = m != -INFINITY ? w / sum * a.rs : 0.f;
    }
  }
}

template <typename E, int TT>
static cudaError_t launch_route16(const RouteArgs16& r, cudaStream_t st) {
  // the row lanes' sums; later the keys and the items' sums
  const int red = 16 * TT * 4 * 64 * 4, fin = TT * r.p.ep * 4 + std::max(kRThreads, TT * r.p.ep / 4) * 16;
  const int smem = std::max(r.a.W_r ? red : 0, fin);
  static std::atomic<bool> done[kMaxDevices] = {};
  const cudaError_t e = set_smem_once((const void*)k_l16_route<E, TT>, 160 * 1024, done);
  if (e != cudaSuccess) return e;
  const bool routes = r.a.W_r || r.a.logits;
  const dim3 grid(r.a.W_r ? r.p.ks : 1, r.a.W_r ? r.p.et : 1, routes ? r.p.z : 1);
  note_launch();
  return launch_pdl(k_l16_route<E, TT>, grid, dim3(kRThreads), smem, st, r);
}
template <typename E>
static cudaError_t launch_route16(const RouteArgs16& r, cudaStream_t st) {
  switch (r.p.tt) {
    case 1: return launch_route16<E, 1>(r, st);
    case 2: return launch_route16<E, 2>(r, st);
    case 4: return launch_route16<E, 4>(r, st);
    default: return launch_route16<E, 8>(r, st);
  }
}

cudaError_t launch_layer16(const Layer16Args& a, cudaStream_t st) {
  const Layer16Ws w = layer16_ws(a.T, a.H, a.I, a.E, a.k, a.S);
  RouteArgs16 r = {a, route_plan(a.T, a.H, a.E), reinterpret_cast<float*>(a.ws + w.router)};
  const cudaError_t e = a.dtype == MOE_DT_BF16 ? launch_route16<Bf16>(r, st) : launch_route16<F16>(r, st);
  if (e != cudaSuccess) return e;
  FewArgs f = {};
  f.R = a.T; f.K1 = a.H; f.F1 = a.I; f.K2 = a.I; f.F2 = a.H; f.act = a.act; f.dtype = a.dtype; f.status = a.status;
  f.E = a.E; f.k = a.k; f.S = a.S; f.ids = a.ids; f.wts = a.w; f.b1 = a.b1;
  f.y = reinterpret_cast<uint16_t*>(a.ws + w.y); f.ldy = w.ldy;
  f.ticket = reinterpret_cast<int32_t*>(a.ws);
  f.done = f.ticket + 1;
  f.joined = f.ticket + 16;
  f.part = reinterpret_cast<float*>(a.ws + w.part);
  f.out = a.out; f.ldo = a.ldo;
  return launch_few_layer(f, a.x, a.ldx, a.w1, a.g1, a.ld1, a.w2, a.g2, a.ld2, st);
}

}  // namespace moe
