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
// Bound: HBM (per gated element 8 bytes forward, 10 backward). One pass: a
// quarter-warp owns a 128-column block, sixteen columns a lane, so the block's
// largest magnitude takes three shuffles. Aligned rows go from memory to
// registers and back; rows at any alignment cross shared memory both ways. The
// backward adds a row's dw over its quarter-warps in a fixed order. NaN passes
// through every activation; an infinity or NaN becomes a NaN code and leaves
// the block's scale to the others.
// Measured, bf16 SwiGLU, y~ asked for: 65536 x 2880 forward 224 us, backward 280
// (6.7 TB/s each); 16384 x 2048 41 and 53 us; at odd alignments 16385 x 2047 67
// and 79 us (4.0, 4.3 TB/s: the shifts of both directions, about half the issue
// slots), 65536 x 2881 341 and 414.
#include "blocks.cuh"

namespace moe {

constexpr int kCkptThreads = 256;
constexpr int kCkptQuarters = kCkptThreads / 8;

// 1 / (1 + 2^(-v log2 e)): the exponential and the reciprocal on the
// special-function unit, relative error about 2^-22 each; the rounding of the
// exponent adds |v| 2^-24, 2^-17 at most where 2^x is finite. Together below
// the half step of the 16 bits that leave here (2^-9, 2^-12). Past the
// exponent's range 2^x is 0 or infinity and the quotient 1 or 0. NaN stays NaN.
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

// Half a row's block forward: y's words, codes and scales.
template <typename E, int ACT, bool FIN>
__device__ __forceinline__ void fwd16(uint32_t (&y)[8], uint32_t (&cg)[4], uint32_t (&cu)[4], const uint32_t (&gw)[8],
                                      const uint32_t (&uw)[8], float sg, float su, float w, const ActParams& p) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 g = pair_of<E>(gw[j]), u = pair_of<E>(uw[j]);
    y[j] = E::from2(w * ckpt_act<ACT, FIN>(g.x, u.x, p), w * ckpt_act<ACT, FIN>(g.y, u.y, p));
  }
  codes16<E, FIN>(cg, gw, 1.0f / sg);
  if constexpr (ACT != MOE_ACT_SRELU) codes16<E, FIN>(cu, uw, 1.0f / su);
}

// A block's scales and their codes, and y: the words of both halves to the
// words of y and the codes.
template <typename E, int ACT>
__device__ __forceinline__ void fwd_block(uint32_t (&y)[8], uint32_t (&cg)[4], uint32_t (&cu)[4], float& sg, float& su,
                                          const uint32_t (&gw)[8], const uint32_t (&uw)[8], float w, const ActParams& p,
                                          unsigned lanes) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
  // both halves' largest magnitudes in one word: three shuffles
  uint32_t mm = mag_bits(gw) | (GATED ? mag_bits(uw) << 16 : 0u);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) mm = __vmaxu2(mm, __shfl_xor_sync(lanes, mm, o));
  if ((mm & 0xffffu) < E::kInf && (mm >> 16) < E::kInf) {
    sg = block_scale(E::to((uint16_t)(mm & 0xffffu)));
    su = block_scale(E::to((uint16_t)(mm >> 16)));
    fwd16<E, ACT, true>(y, cg, cu, gw, uw, sg, su, w, p);
  } else {
    sg = finite_scale<E>(gw, lanes);
    su = GATED ? finite_scale<E>(uw, lanes) : 1.f;
    fwd16<E, ACT, false>(y, cg, cu, gw, uw, sg, su, w, p);
  }
}

// qpr quarter-warps of a CTA (a power of two) share a row; the others take
// other rows.
template <typename E, int ACT>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_fwd(CkptArgs a, int qpr) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
  pdl_enter();
  const int l = threadIdx.x & 7, qw = threadIdx.x >> 3;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int rpc = kCkptQuarters / qpr, rl = qw / qpr, part = qw % qpr;
  for (int64_t row = (int64_t)blockIdx.x * rpc + rl; row < a.R; row += (int64_t)gridDim.x * rpc) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(a.h) + row * a.ldh;
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy;
    uint8_t* q = a.q + row * a.ldq;
    float* s = a.s + row * nb * (GATED ? 2 : 1);
    const float w = a.w ? a.w[row] : 1.f;
    for (int b = part; b < nb; b += qpr) {
      const int c0 = b * kQBlock, n = min(kQBlock, a.I - c0);
      uint32_t gw[8], uw[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, yw[8], cg[4], cu[4];
      load16(gw, h + c0, l, n);
      if constexpr (GATED) load16(uw, h + a.I + c0, l, n);
      float sg, su;
      fwd_block<E, ACT>(yw, cg, cu, sg, su, gw, uw, w, a.act, lanes);
      store_codes(q + c0, cg, l, n);
      if constexpr (GATED) store_codes(q + a.I + c0, cu, l, n);
      if (l == 0) {
        s[b] = sg;
        if constexpr (GATED) s[nb + b] = su;
      }
      store16(y + c0, yw, l, n);
    }
  }
}

// The same for rows at any alignment. A quarter-warp fetches its next block's
// units into shared memory while it works on one, and its outputs leave
// through shared memory, in whole units.
template <typename E, int ACT>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_fwd_any(CkptArgs a, int qpr) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
  __shared__ __align__(16) uint8_t in_smem[kCkptQuarters][2][(GATED ? 2 : 1) * kStageBytes];
  __shared__ __align__(16) uint8_t out_smem[kCkptQuarters][kStageBytes];
  static_assert(kCodeBytes <= kStageBytes, "either fits");
  pdl_enter();
  const int l = threadIdx.x & 7, qw = threadIdx.x >> 3;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int rpc = kCkptQuarters / qpr, rl = qw / qpr, part = qw % qpr;
  const int64_t step = (int64_t)gridDim.x * rpc;
  const uint8_t* h0 = reinterpret_cast<const uint8_t*>(a.h);
  uint8_t* out = out_smem[qw];
  auto fetch = [&](int64_t row, int b, int stage) {
    if (row < a.R && b < nb) {
      const uint8_t* h = h0 + row * a.ldh * 2;
      fetch_block<2>(in_smem[qw][stage], h, b * kQBlock, a.I, h0, l);
      if constexpr (GATED) fetch_block<2>(in_smem[qw][stage] + kStageBytes, h + 2 * (int64_t)a.I, b * kQBlock, a.I, h0, l);
    }
    cp_async_commit();
  };
  int stage = 0;
  int64_t row = (int64_t)blockIdx.x * rpc + rl;
  fetch(row, part, 0);
  for (; row < a.R; row += step) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(a.h) + row * a.ldh;
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy;
    uint8_t* q = a.q + row * a.ldq;
    float* s = a.s + row * nb * (GATED ? 2 : 1);
    const float w = a.w ? a.w[row] : 1.f;
    for (int b = part; b < nb; b += qpr, stage ^= 1) {
      const int c0 = b * kQBlock, n = min(kQBlock, a.I - c0);
      const bool more = b + qpr < nb;
      fetch(more ? row : row + step, more ? b + qpr : part, stage ^ 1);
      cp_async_wait<1>();
      __syncwarp(lanes);
      uint32_t gw[8], uw[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, yw[8], cg[4], cu[4];
      const uint8_t* in = in_smem[qw][stage];
      read16(gw, in, (int)((uintptr_t)(h + c0) & 15), l);
      if constexpr (GATED) read16(uw, in + kStageBytes, (int)((uintptr_t)(h + a.I + c0) & 15), l);
      float sg, su;
      fwd_block<E, ACT>(yw, cg, cu, sg, su, gw, uw, w, a.act, lanes);
      auto put_codes = [&](uint8_t* p, const uint32_t(&v)[4]) {
        stage_codes(out, v, l);
        __syncwarp(lanes);
        store_staged_codes(p, out, l, n);
        __syncwarp(lanes);
      };
      put_codes(q + c0, cg);
      if constexpr (GATED) put_codes(q + a.I + c0, cu);
      if (l == 0) {
        s[b] = sg;
        if constexpr (GATED) s[nb + b] = su;
      }
      stage16(out, y + c0, yw, l);
      __syncwarp(lanes);
      store_staged(y + c0, out, l, n);
      __syncwarp(lanes);
    }
  }
  cp_async_wait<0>();
}

__device__ __forceinline__ bool nan_code(uint32_t w) {      // a byte whose low seven bits are all set
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
}

// Sixteen columns backward: the words of dh's halves and of y; returns the
// lane's part of dw. Columns past the row's end are zeros and add nothing.
template <typename E, int ACT, bool FIN>
__device__ __forceinline__ float bwd16(uint32_t (&dg)[8], uint32_t (&du)[8], uint32_t (&y)[8], const uint32_t (&qg)[4],
                                       const uint32_t (&qu)[4], const uint32_t (&dw_)[8], float sg, float su, float w,
                                       const ActParams& p) {
  float dw = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 g = e4m3x2_to_f32x2((uint16_t)(qg[j >> 1] >> (16 * (j & 1))));
    const float2 u = e4m3x2_to_f32x2((uint16_t)(qu[j >> 1] >> (16 * (j & 1))));
    const float2 d = pair_of<E>(dw_[j]);
    const float3 fx = ckpt_act_grad<ACT, FIN>(g.x * sg, u.x * su, p);
    const float3 fy = ckpt_act_grad<ACT, FIN>(g.y * sg, u.y * su, p);
    dw = fmaf(d.x, fx.x, dw);
    dw = fmaf(d.y, fy.x, dw);
    const float wx = w * d.x, wy = w * d.y;
    y[j] = E::from2(w * fx.x, w * fy.x);
    dg[j] = E::from2(wx * fx.y, wy * fy.y);
    if constexpr (ACT != MOE_ACT_SRELU) du[j] = E::from2(wx * fx.z, wy * fy.z);
  }
  return dw;
}

// The row's dw from its quarter-warps' parts, in a fixed order. WARP: the row's
// quarters are of one warp; otherwise of the CTA (sdw: two rounds' parts).
template <bool WARP>
__device__ __forceinline__ void join_dw(float* out, float dw, bool live, int part, int qpr, float* sdw, int qw, int l) {
  __syncwarp();
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) dw += __shfl_xor_sync(kFull, dw, o);
  if constexpr (WARP) {
    if (qpr > 1) dw += __shfl_xor_sync(kFull, dw, 8);
    if (qpr > 2) dw += __shfl_xor_sync(kFull, dw, 16);
    if (live && part == 0 && l == 0) *out = dw;
  } else {
    if (l == 0) sdw[qw] = dw;
    __syncthreads();
    if (live && part == 0 && l == 0) {
      float t = 0.f;
      for (int i = 0; i < qpr; ++i) t += sdw[qw + i];
      *out = t;
    }
  }
}

template <typename E, int ACT>
__device__ __forceinline__ float bwd_block(uint32_t (&dg)[8], uint32_t (&du)[8], uint32_t (&y)[8], const uint32_t (&qg)[4],
                                           const uint32_t (&qu)[4], const uint32_t (&d)[8], float sg, float su, float w,
                                           const ActParams& p) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) nan |= nan_code(qg[j]) | nan_code(qu[j]);
  // 448 s overflows for the largest scales; a caller's scale may be anything
  const bool fin = !nan && fabsf(sg) < 1e35f && fabsf(su) < 1e35f;
  return fin ? bwd16<E, ACT, true>(dg, du, y, qg, qu, d, sg, su, w, p)
             : bwd16<E, ACT, false>(dg, du, y, qg, qu, d, sg, su, w, p);
}

// qpr quarter-warps of a CTA share a row, whose dw crosses shared memory.
template <typename E, int ACT>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_bwd(CkptArgs a, int qpr) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
  pdl_enter();
  __shared__ float sdw[2][kCkptQuarters];
  const int l = threadIdx.x & 7, qw = threadIdx.x >> 3;
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int rpc = kCkptQuarters / qpr, rl = qw / qpr, part = qw % qpr;     // rows a CTA takes
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
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy;
      for (int b = part; b < nb; b += qpr) {
        const int c0 = b * kQBlock, n = min(kQBlock, a.I - c0);
        uint32_t qg[4], qu[4] = {0u, 0u, 0u, 0u}, d[8], dg[8], du[8], yw[8];
        load_codes(qg, q + c0, l, n);
        if constexpr (GATED) load_codes(qu, q + a.I + c0, l, n);
        load16(d, dy + c0, l, n);
        dw += bwd_block<E, ACT>(dg, du, yw, qg, qu, d, s[b], GATED ? s[nb + b] : 0.f, w, a.act);
        store16(dh + c0, dg, l, n);
        if constexpr (GATED) store16(dh + a.I + c0, du, l, n);
        if (a.y) store16(y + c0, yw, l, n);
      }
    }
    if (a.dw) join_dw<false>(a.dw + row, dw, live, part, qpr, sdw[flip], qw, l);
  }
}

// The same for rows at any alignment. WARP: at most four quarter-warps, of one
// warp, share a row: its dw needs shuffles only, and warps go on at their own
// pace. A quarter-warp fetches its next block's units into shared memory while
// it works on one (16385 x 2047 79 us; with loads of its own columns, which
// waited 8 of 13 cycles an instruction, 102), and its outputs leave through
// shared memory too (store_staged; from registers 132).
template <typename E, int ACT, bool WARP>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_bwd_any(CkptArgs a, int qpr) {
  constexpr bool GATED = ACT != MOE_ACT_SRELU;
  constexpr int kIn = kStageBytes + (GATED ? 2 : 1) * kCodeBytes;
  __shared__ __align__(16) uint8_t in_smem[kCkptQuarters][2][kIn];
  __shared__ __align__(16) uint8_t out_smem[kCkptQuarters][kStageBytes];
  __shared__ float sdw[2][WARP ? 1 : kCkptQuarters];
  pdl_enter();
  const int l = threadIdx.x & 7, qc = threadIdx.x >> 3, qw = WARP ? qc & 3 : qc;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  const int nb = (a.I + kQBlock - 1) / kQBlock;
  const int rpg = (WARP ? 4 : kCkptQuarters) / qpr, rl = qw / qpr, part = qw % qpr;   // rows a warp (CTA) takes
  const int64_t group = WARP ? (int64_t)blockIdx.x * (kCkptThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = (WARP ? (int64_t)gridDim.x * (kCkptThreads / 32) : gridDim.x) * rpg;
  const uint8_t* dy0 = reinterpret_cast<const uint8_t*>(a.dy);
  uint8_t* out = out_smem[qc];
  float sg_next = 0.f, su_next = 0.f;
  auto fetch = [&](int64_t row, int b, int stage) {
    if (row < a.R && b < nb) {
      uint8_t* in = in_smem[qc][stage];
      const uint8_t* q = a.q + row * a.ldq;
      const float* s = a.s + row * nb * (GATED ? 2 : 1);
      fetch_block<2>(in, dy0 + row * a.lddy * 2, b * kQBlock, a.I, dy0, l);
      fetch_block<1>(in + kStageBytes, q, b * kQBlock, a.I, a.q, l);
      if constexpr (GATED) fetch_block<1>(in + kStageBytes + kCodeBytes, q + a.I, b * kQBlock, a.I, a.q, l);
      sg_next = s[b];
      if constexpr (GATED) su_next = s[nb + b];
    }
    cp_async_commit();
  };
  int flip = 0, stage = 0;
  fetch(group * rpg + rl, part, 0);
  for (int64_t r0 = group * rpg; r0 < a.R; r0 += step, flip ^= 1) {
    const int64_t row = r0 + rl;
    const bool live = row < a.R;
    const float w = live && a.w ? a.w[row] : 1.f;
    float dw = 0.f;
    if (live) {
      const uint8_t* q = a.q + row * a.ldq;
      const uint16_t* dy = reinterpret_cast<const uint16_t*>(a.dy) + row * a.lddy;
      uint16_t* dh = reinterpret_cast<uint16_t*>(a.dh) + row * a.lddh;
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy;
      for (int b = part; b < nb; b += qpr, stage ^= 1) {
        const int c0 = b * kQBlock, n = min(kQBlock, a.I - c0);
        const float sg = sg_next, su = su_next;
        const bool more = b + qpr < nb;
        fetch(more ? row : row + step, more ? b + qpr : part, stage ^ 1);
        cp_async_wait<1>();
        __syncwarp(lanes);
        uint32_t qg[4], qu[4] = {0u, 0u, 0u, 0u}, d[8], dg[8], du[8], yw[8];
        const uint8_t* in = in_smem[qc][stage];
        read16(d, in, (int)((uintptr_t)(dy + c0) & 15), l);
        read_codes(qg, in + kStageBytes, (int)((uintptr_t)(q + c0) & 15), l);
        if constexpr (GATED) read_codes(qu, in + kStageBytes + kCodeBytes, (int)((uintptr_t)(q + a.I + c0) & 15), l);
        dw += bwd_block<E, ACT>(dg, du, yw, qg, qu, d, sg, su, w, a.act);
        auto put = [&](uint16_t* p, const uint32_t(&v)[8]) {
          stage16(out, p, v, l);
          __syncwarp(lanes);
          store_staged(p, out, l, n);
          __syncwarp(lanes);
        };
        put(dh + c0, dg);
        if constexpr (GATED) put(dh + a.I + c0, du);
        if (a.y) put(y + c0, yw);
      }
    }
    if (a.dw) join_dw<WARP>(a.dw + row, dw, live, part, qpr, sdw[flip], qw, l);
  }
  cp_async_wait<0>();
}

// ---- host ----------------------------------------------------------------------
static bool al(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename E, int ACT>
static cudaError_t fwd_t(const CkptArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.ldh % 8 == 0 && a.ldy % 8 == 0 && a.ldq % 8 == 0 && al(a.h, 16) && al(a.y, 16) &&
                   al(a.q, 8);
  const int qpr = quarters_a_row(a.I, kCkptQuarters), rpc = kCkptQuarters / qpr;
  const int64_t g = std::min<int64_t>((a.R + rpc - 1) / rpc, (int64_t)device_sms() * 32);
  note_launch();
  if (vec) return launch_pdl(k_ckpt_fwd<E, ACT>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a, qpr);
  return launch_pdl(k_ckpt_fwd_any<E, ACT>, dim3((unsigned)g), dim3(kCkptThreads), 0, st, a, qpr);
}

template <typename E, int ACT>
static cudaError_t bwd_t(const CkptArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.lddy % 8 == 0 && a.lddh % 8 == 0 && a.ldq % 8 == 0 && al(a.dy, 16) &&
                   al(a.dh, 16) && al(a.q, 8) && (!a.y || (a.ldy % 8 == 0 && al(a.y, 16)));
  // A warp a row (or more rows) at odd alignments, where that leaves a warp
  // several rows: 16385 x 2047 79.6 us (87.2 by CTAs), 65536 x 2881 414 (445);
  // with fewer rows the last ones leave SMs idle (5000 x 2047 31.1 and 27.2).
  // Aligned rows gain nothing (16384 x 2048 53.1 and 52.7, x 2880 76.6 and 72.6).
  const bool warp = !vec && a.R >= 96LL * device_sms();
  const int qpr = quarters_a_row(a.I, warp ? 4 : kCkptQuarters);
  const int64_t rows = kCkptQuarters / qpr;     // a CTA's
  const dim3 g((unsigned)std::min<int64_t>((a.R + rows - 1) / rows, (int64_t)device_sms() * 32)), b(kCkptThreads);
  note_launch();
  if (vec) return launch_pdl(k_ckpt_bwd<E, ACT>, g, b, 0, st, a, qpr);
  if (warp) return launch_pdl(k_ckpt_bwd_any<E, ACT, true>, g, b, 0, st, a, qpr);
  return launch_pdl(k_ckpt_bwd_any<E, ACT, false>, g, b, 0, st, a, qpr);
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
