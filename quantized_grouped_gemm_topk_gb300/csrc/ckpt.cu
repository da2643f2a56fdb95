// The experts' activation with an 8-bit checkpoint of its input.
//
// Forward, from h = W1's output (gate half and up half; sReLU: one half):
//   y = w_row act(g, u) in 16 bits, and h's checkpoint: E4M3 codes q with one
//   fp32 scale s per 128 columns of each half (blocks do not cross the halves).
// Backward, from the checkpoint alone (g~ = s q): with d = w_row dy,
//   dg = d act_g(g~, u~), du = d act_u(g~, u~), dw_row = sum dy act(g~, u~),
//   and, where asked for, y~ = w_row act(g~, u~) again for W2's weight
//   gradient, so neither h nor y is kept in 16 bits between the passes.
//
// Bound: HBM (per gated element 8 bytes forward, 10 backward). One pass, no
// shared memory: a half-warp owns a 128-column block, eight columns a lane
// (one 16-byte access for each half), so the block's largest magnitude takes
// four shuffles. The backward adds a row's dw over its half-warps in a fixed
// order. NaN passes through every activation; an infinity or NaN becomes a
// NaN code and leaves the block's scale to the others.
#include "ops.cuh"

namespace moe {

constexpr int kCkptThreads = 256;
constexpr int kCkptHalfWarps = kCkptThreads / 16;

// max(h, 0) and the clamp with NaN kept (fmaxf / fminf would drop it).
__device__ __forceinline__ float relu_nan(float h) { return h <= 0.f ? 0.f : h; }
__device__ __forceinline__ float clamp_nan(float v, float lim) { return v < -lim ? -lim : (v > lim ? lim : v); }

// Phi(v) by erfc: 1 + erf(v) would lose every digit where v is far below zero.
__device__ __forceinline__ float ckpt_cdf(float v) { return 0.5f * erfcf(v * -0.70710678118654752f); }

__device__ __forceinline__ float ckpt_act(float g, float u, const ActParams& p) {
  if (p.act == MOE_ACT_SRELU) {
    const float r = relu_nan(g);
    return r * r;
  }
  if (p.act == MOE_ACT_SWIGLU) return g * sigmoidf_(g) * u;
  if (p.act == MOE_ACT_GEGLU) return g * ckpt_cdf(g) * u;
  const float gc = clamp_nan(g, p.limit), uc = clamp_nan(u, p.limit);
  return gc * sigmoidf_(p.alpha * gc) * uc;
}

// (act, d act / dg, d act / du)
__device__ __forceinline__ float3 ckpt_act_grad(float g, float u, const ActParams& p) {
  if (p.act == MOE_ACT_SRELU) {
    const float r = relu_nan(g);
    return make_float3(r * r, 2.f * r, 0.f);
  }
  if (p.act == MOE_ACT_SWIGLU) {
    const float s = sigmoidf_(g), gs = g * s;
    return make_float3(gs * u, (s + gs * (1.0f - s)) * u, gs);
  }
  if (p.act == MOE_ACT_GEGLU) {
    const float c = ckpt_cdf(g), gc = g * c;
    return make_float3(gc * u, (c + g * normal_pdf(g)) * u, gc);
  }
  const float gc = clamp_nan(g, p.limit), uc = clamp_nan(u, p.limit);
  const float s = sigmoidf_(p.alpha * gc), gs = gc * s;
  // the gradient stops outside the clamp; NaN compares as inside and is kept
  const float dg = fabsf(g) > p.limit ? 0.f : (s + p.alpha * gs * (1.0f - s)) * uc;
  const float du = fabsf(u) > p.limit ? 0.f : gs;
  return make_float3(gs * uc, dg, du);
}

// The lane's eight columns of a 128-column block, at c0 + lane16 * 8 + j
// (VEC: 16-byte accesses, I a multiple of 8) or c0 + lane16 + 16 j; columns
// past n read as zero.
template <bool VEC>
__device__ __forceinline__ int col_of(int l, int j) { return VEC ? l * 8 + j : l + 16 * j; }

template <typename E, bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const typename E::raw* p, int l, int n) {
  if constexpr (VEC) {
    Pack<E, 8> k;
    if (l * 8 < n) load_pack(k, p + l * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = l * 8 < n ? E::to(k.v[j]) : 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = l + 16 * j < n ? E::to(p[l + 16 * j]) : 0.f;
  }
}
template <typename E, bool VEC>
__device__ __forceinline__ void store8(typename E::raw* p, const float (&v)[8], int l, int n) {
  if constexpr (VEC) {
    Pack<E, 8> k;
#pragma unroll
    for (int j = 0; j < 8; ++j) k.v[j] = E::from(v[j]);
    if (l * 8 < n) store_pack<E, 8>(p + l * 8, k);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (l + 16 * j < n) p[l + 16 * j] = E::from(v[j]);
  }
}

template <int W>
__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Codes of one half's block; the lanes of the half-warp agree on the scale.
template <bool VEC>
__device__ __forceinline__ void quant_store8(const float (&v)[8], uint8_t* q, float* s, int l, int n, bool live) {
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, finite_mag(v[j]));
  const float sc = block_scale(half_max<16>(am));
  const float inv = 1.0f / sc;
  uint16_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = f32x2_to_e4m3x2(code_arg(v[2 * j], inv), code_arg(v[2 * j + 1], inv));
  if (!live) return;
  if constexpr (VEC) {
    if (l * 8 < n)
      *reinterpret_cast<uint2*>(q + l * 8) = make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16),
                                                        (uint32_t)c[2] | ((uint32_t)c[3] << 16));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (l + 16 * j < n) q[l + 16 * j] = (uint8_t)(c[j >> 1] >> (8 * (j & 1)));
  }
  if (l == 0) *s = sc;
}

template <bool VEC>
__device__ __forceinline__ void dequant8(float (&v)[8], const uint8_t* q, float s, int l, int n) {
  if constexpr (VEC) {
    uint2 w = make_uint2(0u, 0u);
    if (l * 8 < n) w = *reinterpret_cast<const uint2*>(q + l * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = e4m3x2_to_f32x2((uint16_t)((j < 2 ? w.x : w.y) >> (16 * (j & 1))));
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = l + 16 * j < n ? e4m3_to_f32(q[l + 16 * j]) * s : 0.f;
  }
}

template <typename E, bool VEC, bool GATED>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_fwd(CkptArgs a) {
  using raw = typename E::raw;
  pdl_enter();
  const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int64_t items = a.R * nb;
  // both half-warps of a warp go round together: the shuffles need them
  const int64_t step = (int64_t)gridDim.x * kCkptHalfWarps;
  for (int64_t it0 = (int64_t)blockIdx.x * kCkptHalfWarps + (hw & ~1); it0 < items; it0 += step) {
    const int64_t it = it0 + (hw & 1);
    const bool live = it < items;
    const int64_t row = live ? it / nb : 0;
    const int b = live ? (int)(it - row * nb) : 0, c0 = b * kQBlock, n = live ? min(kQBlock, a.I - c0) : 0;
    const raw* h = reinterpret_cast<const raw*>(a.h) + row * a.ldh + c0;
    uint8_t* q = a.q + row * a.ldq + c0;
    float* s = a.s + row * nb * (GATED ? 2 : 1) + b;
    float g[8], u[8], y[8];
    load8<E, VEC>(g, h, l, n);
    if constexpr (GATED) load8<E, VEC>(u, h + a.I, l, n);
    const float w = a.w && live ? a.w[row] : 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = w * ckpt_act(g[j], GATED ? u[j] : 0.f, a.act);
    quant_store8<VEC>(g, q, s, l, n, live);
    if constexpr (GATED) quant_store8<VEC>(u, q + a.I, s + nb, l, n, live);
    store8<E, VEC>(reinterpret_cast<raw*>(a.y) + row * a.ldy + c0, y, l, n);
  }
}

// hpr half-warps of a CTA (a power of two, at least two for more than one
// block) share a row; the others take other rows.
template <typename E, bool VEC, bool GATED>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_bwd(CkptArgs a, int hpr) {
  using raw = typename E::raw;
  pdl_enter();
  __shared__ float sdw[2][kCkptHalfWarps];
  const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int rpc = kCkptHalfWarps / hpr, rl = hw / hpr, part = hw % hpr;
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * rpc; r0 < a.R; r0 += (int64_t)gridDim.x * rpc, flip ^= 1) {
    const int64_t row = r0 + rl;
    const bool live = row < a.R;
    const float w = live && a.w ? a.w[row] : 1.f;
    float dw = 0.f;
    if (live) {
      const uint8_t* q = a.q + row * a.ldq;
      const float* s = a.s + row * nb * (GATED ? 2 : 1);
      const raw* dy = reinterpret_cast<const raw*>(a.dy) + row * a.lddy;
      raw* dh = reinterpret_cast<raw*>(a.dh) + row * a.lddh;
      for (int b = part; b < nb; b += hpr) {
        const int c0 = b * kQBlock, n = min(kQBlock, a.I - c0);
        float g[8], u[8], d[8], y[8];
        dequant8<VEC>(g, q + c0, s[b], l, n);
        if constexpr (GATED) dequant8<VEC>(u, q + a.I + c0, s[nb + b], l, n);
        load8<E, VEC>(d, dy + c0, l, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float3 f = ckpt_act_grad(g[j], GATED ? u[j] : 0.f, a.act);
          // columns past the row's end are zeros and add nothing
          dw = fmaf(d[j], f.x, dw);
          y[j] = w * f.x;
          g[j] = w * d[j] * f.y;
          if constexpr (GATED) u[j] = w * d[j] * f.z;
        }
        store8<E, VEC>(dh + c0, g, l, n);
        if constexpr (GATED) store8<E, VEC>(dh + a.I + c0, u, l, n);
        if (a.y) store8<E, VEC>(reinterpret_cast<raw*>(a.y) + row * a.ldy + c0, y, l, n);
      }
    }
    if (a.dw) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) dw += __shfl_xor_sync(kFull, dw, o);
      if (l == 0) sdw[flip][hw] = dw;
      __syncthreads();
      if (live && part == 0 && l == 0) {
        float t = 0.f;
        for (int i = 0; i < hpr; ++i) t += sdw[flip][hw + i];
        a.dw[row] = t;
      }
    }
  }
}

// ---- host ----------------------------------------------------------------------
static bool al(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename E, bool GATED>
static cudaError_t fwd_t(const CkptArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.ldh % 8 == 0 && a.ldy % 8 == 0 && a.ldq % 8 == 0 && al(a.h, 16) && al(a.y, 16) &&
                   al(a.q, 8);
  const int64_t items = a.R * ((a.I + kQBlock - 1) / kQBlock);
  const int64_t g = std::min<int64_t>((items + kCkptHalfWarps - 1) / kCkptHalfWarps, (int64_t)device_sms() * 32);
  note_launch();
  if (vec) return launch_pdl(k_ckpt_fwd<E, true, GATED>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a);
  return launch_pdl(k_ckpt_fwd<E, false, GATED>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a);
}

template <typename E, bool GATED>
static cudaError_t bwd_t(const CkptArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.lddy % 8 == 0 && a.lddh % 8 == 0 && a.ldq % 8 == 0 && al(a.dy, 16) &&
                   al(a.dh, 16) && al(a.q, 8) && (!a.y || (a.ldy % 8 == 0 && al(a.y, 16)));
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  int hpr = 1;
  while (hpr < kCkptHalfWarps && hpr < nb) hpr *= 2;
  const int rpc = kCkptHalfWarps / hpr;
  const int64_t g = std::min<int64_t>((a.R + rpc - 1) / rpc, (int64_t)device_sms() * 32);
  note_launch();
  if (vec) return launch_pdl(k_ckpt_bwd<E, true, GATED>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a, hpr);
  return launch_pdl(k_ckpt_bwd<E, false, GATED>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a, hpr);
}

cudaError_t launch_ckpt_fwd(const CkptArgs& a, cudaStream_t st) {
  const bool gated = a.act.act != MOE_ACT_SRELU;
  if (a.dtype == MOE_DT_F16) return gated ? fwd_t<F16, true>(a, st) : fwd_t<F16, false>(a, st);
  return gated ? fwd_t<Bf16, true>(a, st) : fwd_t<Bf16, false>(a, st);
}
cudaError_t launch_ckpt_bwd(const CkptArgs& a, cudaStream_t st) {
  const bool gated = a.act.act != MOE_ACT_SRELU;
  if (a.dtype == MOE_DT_F16) return gated ? bwd_t<F16, true>(a, st) : bwd_t<F16, false>(a, st);
  return gated ? bwd_t<Bf16, true>(a, st) : bwd_t<Bf16, false>(a, st);
}

}  // namespace moe
