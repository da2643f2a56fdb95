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

// 1 / (1 + 2^(-v log2 e)): the exponential and the reciprocal on the
// special-function unit (relative error about 2^-22 each, far below the 16
// bits that leave here); past the exponent's range 2^x is 0 or infinity and
// the quotient 1 or 0. NaN stays NaN.
__device__ __forceinline__ float fast_sigmoid(float v) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
// Phi(v) by erfc: 1 + erf(v) would lose every digit where v is far below zero.
__device__ __forceinline__ float ckpt_cdf(float v) { return 0.5f * erfcf(v * -0.70710678118654752f); }

// The clamp and max(h, 0). FIN: v is known to be finite; otherwise NaN is
// kept, which fminf / fmaxf would drop.
template <bool FIN>
__device__ __forceinline__ float clamp_to(float v, float lim) {
  if (FIN) return fminf(fmaxf(v, -lim), lim);
  return v < -lim ? -lim : (v > lim ? lim : v);
}
template <bool FIN>
__device__ __forceinline__ float relu(float v) {
  if (FIN) return fmaxf(v, 0.f);
  return v <= 0.f ? 0.f : v;
}

template <int ACT, bool FIN>
__device__ __forceinline__ float ckpt_act(float g, float u, const ActParams& p) {
  if constexpr (ACT == MOE_ACT_SRELU) {
    const float r = relu<FIN>(g);
    return r * r;
  } else if constexpr (ACT == MOE_ACT_SWIGLU) {
    return g * fast_sigmoid(g) * u;
  } else if constexpr (ACT == MOE_ACT_GEGLU) {
    return g * ckpt_cdf(g) * u;
  } else {
    const float gc = clamp_to<FIN>(g, p.limit), uc = clamp_to<FIN>(u, p.limit);
    return gc * fast_sigmoid(p.alpha * gc) * uc;
  }
}

// (act, d act / dg, d act / du)
template <int ACT, bool FIN>
__device__ __forceinline__ float3 ckpt_act_grad(float g, float u, const ActParams& p) {
  if constexpr (ACT == MOE_ACT_SRELU) {
    const float r = relu<FIN>(g);
    return make_float3(r * r, 2.f * r, 0.f);
  } else if constexpr (ACT == MOE_ACT_SWIGLU) {
    const float s = fast_sigmoid(g), gs = g * s;
    return make_float3(gs * u, fmaf(gs, 1.0f - s, s) * u, gs);
  } else if constexpr (ACT == MOE_ACT_GEGLU) {
    const float c = ckpt_cdf(g), gc = g * c;
    return make_float3(gc * u, (c + g * normal_pdf(g)) * u, gc);
  } else {
    const float gc = clamp_to<FIN>(g, p.limit), uc = clamp_to<FIN>(u, p.limit);
    const float s = fast_sigmoid(p.alpha * gc), gs = gc * s;
    // the gradient stops outside the clamp, where the clamp changed the value
    // (NaN differs from itself; it is kept)
    const float dg = (gc == g || !FIN && g != g) ? fmaf(p.alpha * gs, 1.0f - s, s) * uc : 0.f;
    const float du = (uc == u || !FIN && u != u) ? gs : 0.f;
    return make_float3(gs * uc, dg, du);
  }
}

// A lane's eight columns of a 128-column block as four words of two 16-bit
// elements: columns 8 l .. 8 l + 7 (VEC: one 16-byte access, I a multiple of
// 8), or l + 16 j. Columns past the block's n are zeros and not written.
template <bool VEC>
__device__ __forceinline__ void load8(uint32_t (&w)[4], const uint16_t* p, int l, int n) {
  if constexpr (VEC) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (l * 8 < n) v = *reinterpret_cast<const uint4*>(p + l * 8);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    uint16_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = l + 16 * j < n ? p[l + 16 * j] : (uint16_t)0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (uint32_t)e[2 * j] | ((uint32_t)e[2 * j + 1] << 16);
  }
}
template <typename E>
__device__ __forceinline__ void unpack8(float (&v)[8], const uint32_t (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = E::to((uint16_t)(w[j] & 0xffffu));
    v[2 * j + 1] = E::to((uint16_t)(w[j] >> 16));
  }
}
template <typename E, bool VEC>
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], int l, int n) {
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
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* q, const uint16_t (&c)[4], int l, int n) {
  if constexpr (VEC) {
    if (l * 8 < n)
      *reinterpret_cast<uint2*>(q + l * 8) = make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16),
                                                        (uint32_t)c[2] | ((uint32_t)c[3] << 16));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (l + 16 * j < n) q[l + 16 * j] = (uint8_t)(c[j >> 1] >> (8 * (j & 1)));
  }
}

// Magnitude bits (16-bit elements without their sign order as integers:
// finite < infinity < NaN) of the largest of the lane's eight.
__device__ __forceinline__ uint32_t mag_bits(const uint32_t (&w)[4]) {
  constexpr uint32_t k = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(w[0] & k, w[1] & k), __vmaxu2(w[2] & k, w[3] & k));
  return max(m & 0xffffu, m >> 16);
}

// E4M3 codes of v at 1 / inv; FIN: without the test for infinities.
template <bool FIN>
__device__ __forceinline__ void codes8(uint16_t (&c)[4], const float (&v)[8], float inv) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = FIN ? f32x2_to_e4m3x2(v[2 * j] * inv, v[2 * j + 1] * inv)
               : f32x2_to_e4m3x2(code_arg(v[2 * j], inv), code_arg(v[2 * j + 1], inv));
}

// The block's scale where some element is an infinity or NaN: the largest of
// the finite ones, over the half-warp.
__device__ __forceinline__ float finite_scale(const float (&v)[8], unsigned half) {
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, finite_mag(v[j]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(half, am, o));
  return block_scale(am);
}

template <typename E, bool VEC, int ACT>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_fwd(CkptArgs a) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
  pdl_enter();
  const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const unsigned half = 0xffffu << (threadIdx.x & 16);
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int64_t items = a.R * nb;
  // both half-warps of a warp go round together (the shuffles need them); the
  // item's row and block are carried along instead of divided out
  const int64_t step = (int64_t)gridDim.x * kCkptHalfWarps;
  const int64_t step_row = step / nb;
  const int step_b = (int)(step - step_row * nb);
  const int64_t it1 = (int64_t)blockIdx.x * kCkptHalfWarps + hw;
  int64_t row_at = it1 / nb;
  int b_at = (int)(it1 - row_at * nb);
  for (int64_t it0 = it1 - (hw & 1); it0 < items; it0 += step) {
    const bool live = it0 + (hw & 1) < items;
    const int64_t row = live ? row_at : 0;
    const int b = live ? b_at : 0, c0 = b * kQBlock, n = live ? min(kQBlock, a.I - c0) : 0;
    row_at += step_row;
    b_at += step_b;
    if (b_at >= nb) {
      b_at -= nb;
      ++row_at;
    }
    const uint16_t* h = reinterpret_cast<const uint16_t*>(a.h) + row * a.ldh + c0;
    uint8_t* q = a.q + row * a.ldq + c0;
    float* s = a.s + row * nb * (GATED ? 2 : 1) + b;
    uint32_t gw[4], uw[4] = {0u, 0u, 0u, 0u};
    load8<VEC>(gw, h, l, n);
    if constexpr (GATED) load8<VEC>(uw, h + a.I, l, n);
    const float w = a.w && live ? a.w[row] : 1.f;
    // both halves' largest magnitudes in one word: four shuffles
    uint32_t mm = mag_bits(gw) | (GATED ? mag_bits(uw) << 16 : 0u);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mm = __vmaxu2(mm, __shfl_xor_sync(kFull, mm, o));
    float g[8], u[8], y[8];
    unpack8<E>(g, gw);
    unpack8<E>(u, uw);
    uint16_t cg[4], cu[4];
    float sg, su;
    if ((mm & 0xffffu) < E::kInf && (mm >> 16) < E::kInf) {
      sg = block_scale(E::to((uint16_t)(mm & 0xffffu)));
      su = block_scale(E::to((uint16_t)(mm >> 16)));
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = w * ckpt_act<ACT, true>(g[j], u[j], a.act);
      codes8<true>(cg, g, 1.0f / sg);
      if constexpr (GATED) codes8<true>(cu, u, 1.0f / su);
    } else {
      sg = finite_scale(g, half);
      su = GATED ? finite_scale(u, half) : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = w * ckpt_act<ACT, false>(g[j], u[j], a.act);
      codes8<false>(cg, g, 1.0f / sg);
      if constexpr (GATED) codes8<false>(cu, u, 1.0f / su);
    }
    __syncwarp();
    store_codes<VEC>(q, cg, l, n);
    if constexpr (GATED) store_codes<VEC>(q + a.I, cu, l, n);
    if (live && l == 0) {
      s[0] = sg;
      if constexpr (GATED) s[nb] = su;
    }
    store8<E, VEC>(reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + c0, y, l, n);
  }
}

// The lane's eight codes of a block, as two words; whether one is NaN.
template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t* q, int l, int n) {
  uint2 w = make_uint2(0u, 0u);
  if constexpr (VEC) {
    if (l * 8 < n) w = *reinterpret_cast<const uint2*>(q + l * 8);
  } else {
    uint8_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = l + 16 * j < n ? q[l + 16 * j] : (uint8_t)0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w.x |= (uint32_t)e[j] << (8 * j);
      w.y |= (uint32_t)e[4 + j] << (8 * j);
    }
  }
  return w;
}
__device__ __forceinline__ bool nan_code(uint2 w) {      // a byte whose low seven bits are all set
  constexpr uint32_t k = 0x7f7f7f7fu;
  return ((((w.x & k) + 0x01010101u) | ((w.y & k) + 0x01010101u)) & 0x80808080u) != 0u;
}
__device__ __forceinline__ void dequant8(float (&v)[8], uint2 w, float s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = e4m3x2_to_f32x2((uint16_t)((j < 2 ? w.x : w.y) >> (16 * (j & 1))));
    v[2 * j] = f.x * s;
    v[2 * j + 1] = f.y * s;
  }
}

// g, u -> dh's halves in place, y; returns the lane's part of dw. Columns past
// the row's end are zeros and add nothing.
template <int ACT, bool FIN>
__device__ __forceinline__ float grad8(float (&g)[8], float (&u)[8], float (&y)[8], const float (&d)[8], float w,
                                       const ActParams& p) {
  float dw = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float3 f = ckpt_act_grad<ACT, FIN>(g[j], u[j], p);
    const float wd = w * d[j];
    dw = fmaf(d[j], f.x, dw);
    y[j] = w * f.x;
    g[j] = wd * f.y;
    u[j] = wd * f.z;
  }
  return dw;
}

// hpr half-warps of a CTA (a power of two) share a row; the others take other
// rows.
template <typename E, bool VEC, int ACT>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_bwd(CkptArgs a, int hpr) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
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
      const uint16_t* dy = reinterpret_cast<const uint16_t*>(a.dy) + row * a.lddy;
      uint16_t* dh = reinterpret_cast<uint16_t*>(a.dh) + row * a.lddh;
      for (int b = part; b < nb; b += hpr) {
        const int c0 = b * kQBlock, n = min(kQBlock, a.I - c0);
        const uint2 qg = load_codes<VEC>(q + c0, l, n);
        uint2 qu = make_uint2(0u, 0u);
        if constexpr (GATED) qu = load_codes<VEC>(q + a.I + c0, l, n);
        uint32_t dword[4];
        load8<VEC>(dword, dy + c0, l, n);
        const float sg = s[b], su = GATED ? s[nb + b] : 0.f;
        float g[8], u[8], d[8], y[8];
        dequant8(g, qg, sg);
        dequant8(u, qu, su);
        unpack8<E>(d, dword);
        // 448 s overflows for the largest scales; a caller's scale may be anything
        const bool fin = !nan_code(qg) && !nan_code(qu) && fabsf(sg) < 1e35f && fabsf(su) < 1e35f;
        dw += fin ? grad8<ACT, true>(g, u, y, d, w, a.act) : grad8<ACT, false>(g, u, y, d, w, a.act);
        store8<E, VEC>(dh + c0, g, l, n);
        if constexpr (GATED) store8<E, VEC>(dh + a.I + c0, u, l, n);
        if (a.y) store8<E, VEC>(reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + c0, y, l, n);
      }
    }
    if (a.dw) {
      __syncwarp();
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

template <typename E, int ACT>
static cudaError_t fwd_t(const CkptArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.ldh % 8 == 0 && a.ldy % 8 == 0 && a.ldq % 8 == 0 && al(a.h, 16) && al(a.y, 16) &&
                   al(a.q, 8);
  const int64_t items = a.R * ((a.I + kQBlock - 1) / kQBlock);
  const int64_t g = std::min<int64_t>((items + kCkptHalfWarps - 1) / kCkptHalfWarps, (int64_t)device_sms() * 32);
  note_launch();
  if (vec) return launch_pdl(k_ckpt_fwd<E, true, ACT>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a);
  return launch_pdl(k_ckpt_fwd<E, false, ACT>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a);
}

template <typename E, int ACT>
static cudaError_t bwd_t(const CkptArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.lddy % 8 == 0 && a.lddh % 8 == 0 && a.ldq % 8 == 0 && al(a.dy, 16) &&
                   al(a.dh, 16) && al(a.q, 8) && (!a.y || (a.ldy % 8 == 0 && al(a.y, 16)));
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  // half-warps a row: the most that leave at most a tenth of them idle in the
  // row's last round
  int hpr = kCkptHalfWarps;
  while (hpr > 1 && 10 * ((nb + hpr - 1) / hpr * hpr) > 11 * nb) hpr /= 2;
  const int rpc = kCkptHalfWarps / hpr;
  const int64_t g = std::min<int64_t>((a.R + rpc - 1) / rpc, (int64_t)device_sms() * 32);
  note_launch();
  if (vec) return launch_pdl(k_ckpt_bwd<E, true, ACT>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a, hpr);
  return launch_pdl(k_ckpt_bwd<E, false, ACT>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a, hpr);
}

template <typename E, bool FWD>
static cudaError_t by_act(const CkptArgs& a, cudaStream_t st) {
  switch (a.act.act) {
    case MOE_ACT_SWIGLU: return FWD ? fwd_t<E, MOE_ACT_SWIGLU>(a, st) : bwd_t<E, MOE_ACT_SWIGLU>(a, st);
    case MOE_ACT_SWIGLU_CLAMP: return FWD ? fwd_t<E, MOE_ACT_SWIGLU_CLAMP>(a, st) : bwd_t<E, MOE_ACT_SWIGLU_CLAMP>(a, st);
    case MOE_ACT_GEGLU: return FWD ? fwd_t<E, MOE_ACT_GEGLU>(a, st) : bwd_t<E, MOE_ACT_GEGLU>(a, st);
    default: return FWD ? fwd_t<E, MOE_ACT_SRELU>(a, st) : bwd_t<E, MOE_ACT_SRELU>(a, st);
  }
}

cudaError_t launch_ckpt_fwd(const CkptArgs& a, cudaStream_t st) {
  return a.dtype == MOE_DT_F16 ? by_act<F16, true>(a, st) : by_act<Bf16, true>(a, st);
}
cudaError_t launch_ckpt_bwd(const CkptArgs& a, cudaStream_t st) {
  return a.dtype == MOE_DT_F16 ? by_act<F16, false>(a, st) : by_act<Bf16, false>(a, st);
}

}  // namespace moe
