// Internal interfaces of the training-side operators (layer norm, grouped
// 16-bit products, FP8 128-block products, activation checkpoints) between
// their C entry points (api_ops.cu) and the kernel files.
#pragma once
#include "internal.cuh"

namespace moe {

// ---- typed loads and stores ---------------------------------------------------
// Elements of a runtime-chosen type, held as template tags.
struct Bf16 {
  using raw = uint16_t;
  static constexpr uint32_t kInf = 0x7f80u;
  static __device__ __forceinline__ float to(raw v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ raw from(float f) { return f32_to_bf16_bits(f); }
  // two at once, a in the low half
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
struct F16 {
  using raw = uint16_t;
  static constexpr uint32_t kInf = 0x7c00u;
  static __device__ __forceinline__ float to(raw v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ raw from(float f) { return __half_as_ushort(__float2half_rn(f)); }
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
struct F32 {
  using raw = float;
  static __device__ __forceinline__ float to(raw v) { return v; }
  static __device__ __forceinline__ raw from(float f) { return f; }
};

// Two fp32 values to an instruction (add / mul / fma .f32x2).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// V consecutive elements as one access (V * sizeof(raw) is 16, or V is 1).
template <typename E, int V>
struct Pack {
  typename E::raw v[V];
  // elements 2 i and 2 i + 1
  __device__ __forceinline__ f32x2 pair(int i) const { return pack2(E::to(v[2 * i]), E::to(v[2 * i + 1])); }
  __device__ __forceinline__ void set_pair(int i, f32x2 p) {
    const float2 f = unpack2(p);
    if constexpr (sizeof(typename E::raw) == 2) reinterpret_cast<uint32_t*>(v)[i] = E::from2(f.x, f.y);
    else { v[2 * i] = f.x; v[2 * i + 1] = f.y; }
  }
};
template <typename E, int V>
__device__ __forceinline__ void load_pack(Pack<E, V>& p, const typename E::raw* src) {
  if constexpr (V == 1) {
    p.v[0] = *src;
  } else {
    static_assert(sizeof(Pack<E, V>) == 16, "a pack is one 16-byte access");
    *reinterpret_cast<uint4*>(&p) = *reinterpret_cast<const uint4*>(src);
  }
}
template <typename E, int V>
__device__ __forceinline__ void store_pack(typename E::raw* dst, const Pack<E, V>& p) {
  if constexpr (V == 1) *dst = p.v[0];
  else *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(&p);
}

// ---- rows at any alignment ------------------------------------------------------
// Sixteen (eight) bytes of a row that starts anywhere: the aligned units that
// hold them, shifted together. A unit is read whole only where all of it lies
// in the row's bytes [lo, hi); in the row's first and last one the elements
// (ES bytes each) are read one by one, so nothing outside the row is touched.
// Bytes outside the row are zeros.
template <int ES, int N>
__device__ __forceinline__ void load_unit(uint32_t (&w)[N / 4], const uint8_t* q, const uint8_t* lo, const uint8_t* hi) {
  if (q >= lo && q + N <= hi) {
    if constexpr (N == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(q);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      w[0] = v.x; w[1] = v.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) w[i] = 0u;
#pragma unroll
  for (int i = 0; i < N; i += ES) {
    const uint8_t* p = q + i;
    if (p >= lo && p < hi) {
      if constexpr (ES == 4) w[i / 4] = *reinterpret_cast<const uint32_t*>(p);
      else if constexpr (ES == 2) w[i / 4] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p) << (8 * (i & 3));
      else w[i / 4] |= (uint32_t)*p << (8 * (i & 3));
    }
  }
}
// The N bytes from byte `off` of 2 N.
template <int ES, int N>
__device__ __forceinline__ void shift_units(uint32_t (&r)[N / 4], uint32_t (&w)[N / 2], int off) {
  constexpr int W = N / 4;
  if constexpr (W == 4) {
    const bool two = off & 8;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = two ? w[i + 2] : w[i];
  }
  const bool one = off & 4;
#pragma unroll
  for (int i = 0; i <= W; ++i) w[i] = one && i + 1 < 2 * W ? w[i + 1] : w[i];
  if constexpr (ES < 4) {
    const uint32_t sh = (uint32_t)(off & 3) * 8;
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = __funnelshift_r(w[i], w[i + 1], sh);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = w[i];
  }
}
template <int ES, int N>
__device__ __forceinline__ void load_any(uint32_t (&r)[N / 4], const void* at, const void* lo_, const void* hi_) {
  const uint8_t *p = reinterpret_cast<const uint8_t*>(at), *lo = reinterpret_cast<const uint8_t*>(lo_),
                *hi = reinterpret_cast<const uint8_t*>(hi_);
  constexpr int W = N / 4;
  const int off = (int)((uintptr_t)p & (N - 1));
  uint32_t a[W], b[W], w[2 * W];
#pragma unroll
  for (int i = 0; i < W; ++i) a[i] = b[i] = 0u;
  if (p < hi) load_unit<ES, N>(a, p - off, lo, hi);
  if (off && p - off + N < hi) load_unit<ES, N>(b, p - off + N, lo, hi);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    w[i] = a[i];
    w[W + i] = b[i];
  }
  shift_units<ES, N>(r, w, off);
}

// Stores the first n of 16 / ES (ES 2, 4) elements at any element alignment.
template <int ES>
__device__ __forceinline__ void store_any(void* at, const uint32_t (&w)[4], int n) {
  uint8_t* p = reinterpret_cast<uint8_t*>(at);
  const int bytes = n * ES;
  if (((uintptr_t)p & 15) == 0 && bytes >= 16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (ES == 4 || ((uintptr_t)p & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (bytes >= 4 * i + 4) *reinterpret_cast<uint32_t*>(p + 4 * i) = w[i];
      else if (bytes >= 4 * i + 2) *reinterpret_cast<uint16_t*>(p + 4 * i) = (uint16_t)w[i];
    }
  } else {
    if (bytes >= 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t v = __funnelshift_r(w[i], w[i + 1], 16);
      if (bytes >= 4 * i + 6) *reinterpret_cast<uint32_t*>(p + 4 * i + 2) = v;
      else if (bytes >= 4 * i + 4) *reinterpret_cast<uint16_t*>(p + 4 * i + 2) = (uint16_t)v;
    }
    if (bytes >= 16) *reinterpret_cast<uint16_t*>(p + 14) = (uint16_t)(w[3] >> 16);
  }
}
// All 16 bytes at any element alignment.
template <int ES>
__device__ __forceinline__ void store_inner(void* at, const uint32_t (&w)[4]) {
  uint8_t* p = reinterpret_cast<uint8_t*>(at);
  if (((uintptr_t)p & 15) == 0) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (ES == 4 || ((uintptr_t)p & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
  } else {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(p + 4 * i + 2) = __funnelshift_r(w[i], w[i + 1], 16);
    *reinterpret_cast<uint16_t*>(p + 14) = (uint16_t)(w[3] >> 16);
  }
}
// Stores the first n of eight bytes at any address.
__device__ __forceinline__ void store_bytes8(uint8_t* p, uint2 w, int n) {
  if (n >= 8 && ((uintptr_t)p & 3) == 0) {
    reinterpret_cast<uint32_t*>(p)[0] = w.x;
    reinterpret_cast<uint32_t*>(p)[1] = w.y;
  } else if (n >= 8) {
    // an odd address: a byte, words or halves of the rest, and the last bytes
    const int lead = 4 - (int)((uintptr_t)p & 3);      // 1, 2 or 3 bytes to the next word
    uint32_t head = w.x;
    if (lead & 1) {
      *p = (uint8_t)head;
      if (lead == 3) *reinterpret_cast<uint16_t*>(p + 1) = (uint16_t)(head >> 8);
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)head;
    }
    *reinterpret_cast<uint32_t*>(p + lead) = __funnelshift_r(w.x, w.y, 8 * lead);
    const uint32_t rest = w.y >> (8 * lead);           // 4 - lead bytes, at a word's start
    uint8_t* e = p + lead + 4;
    if (lead == 3) {
      *e = (uint8_t)rest;
    } else {
      *reinterpret_cast<uint16_t*>(e) = (uint16_t)rest;
      if (lead == 1) e[2] = (uint8_t)(rest >> 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
  }
}

// Largest magnitude E4M3 holds, and the smallest scale of a 128-block: with
// it an all-zero block, or one of fp32 subnormals, divides by a normal number.
constexpr int kQBlock = 128;
constexpr float kE4m3Inv = 1.0f / 448.0f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

// A block's scale from the largest finite magnitude in it.
__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax * kE4m3Inv, kMinScale); }
// |v| of a finite v, 0 of an infinity or NaN (those become NaN codes and do
// not reach the block's scale).
__device__ __forceinline__ float finite_mag(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.f;
}
// v * inv for the E4M3 conversion; an infinity becomes NaN, as E4M3 has none
// and the saturating conversion would turn it into 448.
__device__ __forceinline__ float code_arg(float v, float inv) {
  return fabsf(v) <= 3.402823466e38f ? v * inv : __int_as_float(0x7fffffff);
}

// ---- layer norm (norm.cu) ------------------------------------------------------
struct NormArgs {
  const void* x; int64_t ldx;
  const void* dy; int64_t lddy;         // backward
  const void* gamma; const void* beta;  // nullable: ones / zeros
  float eps;
  int64_t T; int H;
  int dtype, wdtype;
  void* out; int64_t ldo;               // y, or dx
  float* mean; float* rstd;             // forward: nullable outputs; backward: inputs
  void* dgamma; void* dbeta;            // backward, nullable
  float* part;                          // backward: [P][2][H] partial sums
};
// Rows of partial sums that the backward writes for T x H at most.
constexpr int kNormMaxParts = 1024;
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st);

// ---- activation checkpoints (ckpt.cu) -------------------------------------------
struct CkptArgs {
  const void* h; int64_t ldh;           // forward
  const void* dy; int64_t lddy;         // backward
  const float* w;                       // nullable: ones
  int64_t R; int I;
  int dtype;
  ActParams act;
  void* y; int64_t ldy;                 // backward: nullable
  uint8_t* q; int64_t ldq;              // codes (backward: input)
  float* s;                             // [R][halves * ceil(I / 128)] (backward: input)
  void* dh; int64_t lddh;               // backward
  float* dw;                            // backward, nullable
};
cudaError_t launch_ckpt_fwd(const CkptArgs& a, cudaStream_t st);
cudaError_t launch_ckpt_bwd(const CkptArgs& a, cudaStream_t st);

// ---- 128-block FP8 quantisers (quant128.cu) --------------------------------------
struct QuantRowsArgs {
  const void* x; int64_t ldx; int64_t R; int C; int dtype;
  uint8_t* q; int64_t ldq; float* s; int64_t lds;
};
cudaError_t launch_quant128_rows(const QuantRowsArgs& a, cudaStream_t st);
struct QuantWeightsArgs {
  const void* w; int64_t wg, ldw; int G, N, K; int dtype;
  uint8_t* q; int64_t qg, ldq; float* s;
  uint8_t* qt; int64_t qtg, ldqt; float* st;    // nullable: the transposed copy
};
cudaError_t launch_quant128_weights(const QuantWeightsArgs& a, cudaStream_t st);

// ---- products (gemm16.cu, gemm_fp8.cu) --------------------------------------------
struct MmArgs {
  int R, N, K, G;               // rows; output columns; reduction (wgrad: dW is N x K, reduced over rows)
  const int32_t* offsets;       // [G + 1], nullable: one group of all rows
  const void* a; int64_t lda;   // rows mode: x [R][K]; wgrad: dy [R][N]
  const void* b; int64_t ldb, bg;   // rows mode: w [G][N][K] or, trans_b, [G][K][N]; wgrad: x [R][K]
  int trans_b;
  int dtype;                    // 16-bit operands
  const float* sa; int64_t ldsa;    // FP8: [R][ceil(K / 128)]
  const float* sb;              // FP8: [G][ceil(N / 128)][ceil(K / 128)]
  void* out; int64_t ldo, og;   // rows mode: [R][N]; wgrad: [G][N][K], og between groups
  int out_dtype;
  int32_t* status;
  float* part;                  // fp32 partial sums of a split product
  int S;                        // pieces of the reduction (1: no partial sums)
};
enum { kMmRows = 0, kMmWgrad = 1, kMmFp8 = 2 };
// SMs a tile (a pair or one), widest tile and pieces of the reduction, from the
// sizes alone.
struct MmPlan {
  int cg, bn, S;
};
MmPlan mm_plan(int kind, int R, int N, int K, int G);
int mm_splits(int kind, int R, int N, int K, int G);
// Bytes of partial sums that suffice for any product of at most R rows.
int64_t mm_part_bytes(int kind, int R, int N, int K, int G);
// Adds the partial sums of a split product into out.
cudaError_t launch_mm_join(const MmArgs& a, bool wgrad, cudaStream_t st);
// Tensor map of rank dimensions (innermost first; strides in elements, from
// the second axis on), 128-byte swizzle, zeros past every edge.
bool make_tmap(CUtensorMap* map, const void* base, int esize, int rank, const int64_t* dims, const int64_t* strides,
               const int* box);
cudaError_t launch_mm16(const MmArgs& a, bool wgrad, cudaStream_t st);
cudaError_t launch_mm_fp8(const MmArgs& a, cudaStream_t st);

// ---- dense products with an epilogue (linear.cu) --------------------------------
// Whether an activation takes a gate and an up column.
__host__ __device__ constexpr bool act_gated(int act) { return act < MOE_ACT_SRELU; }
// Phi(v) and exp(-v^2 / 2), of which Phi's density is a multiple. For x >= 0
// Phi(-x) = exp(-x^2 / 2) Q(x), where Q (Mills' ratio times the density's constant) is
// smooth and falls like 1 / x: here t p(t) with t = 1 / (1 + 0.3 x) and p of degree 7,
// fitted for the least relative error (1.5e-7, by iteratively reweighted least
// squares). So small values of negative v keep their digits (1 + erf would cancel):
// off by at most (8 + v^2) / 2 units, most of them the exponential's. CUDA's erfcf and
// expf are as exact and cost four times as much, 5 us of a product of 333 x 2880 x 1984.
__device__ __forceinline__ float2 cdf_exp(float v) {
  const float x = fabsf(v), t = __fdividef(1.f, fmaf(0.3f, x, 1.f)), e = __expf(-0.5f * (v * v));
  float p = 0.03568089008331299f;
  p = fmaf(p, t, -0.1572285145521164f);
  p = fmaf(p, t, 0.2063971906900406f);
  p = fmaf(p, t, -0.05372370406985283f);
  p = fmaf(p, t, 0.12858273088932037f);
  p = fmaf(p, t, 0.09990713000297546f);
  p = fmaf(p, t, 0.12075497210025787f);
  p = fmaf(p, t, 0.11962923407554626f);
  const float q = p * t * e;
  return make_float2(v < 0.f ? q : 1.f - q, e);
}
__device__ __forceinline__ float cdf_(float v) { return cdf_exp(v).x; }
// Phi(v) + v phi(v), the derivative of v Phi(v), and v Phi(v).
__device__ __forceinline__ float2 gelu_grad(float v) {
  const float2 c = cdf_exp(v);
  return make_float2(fmaf(v * 0.39894228040143268f, c.y, c.x), v * c.x);
}
// Clamp to [-lim, lim] that lets a NaN through.
__device__ __forceinline__ float clamp_(float v, float lim) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(lim));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(-lim));
  return v;
}
__device__ __forceinline__ float act_one(float z, int act) {
  if (act == MOE_ACT_SRELU) return z <= 0.f ? 0.f : z * z;
  if (act == MOE_ACT_GELU) return z * cdf_(z);
  if (act == MOE_ACT_SILU) return z * sigmoidf_(z);
  return z;
}
__device__ __forceinline__ float act_two(float g, float u, const ActParams& p) {
  if (p.act == MOE_ACT_SWIGLU) return g * sigmoidf_(g) * u;
  if (p.act == MOE_ACT_GEGLU) return g * cdf_(g) * u;
  const float gc = clamp_(g, p.limit);
  return gc * sigmoidf_(p.alpha * gc) * clamp_(u, p.limit);
}
// d act'(z), and d times the derivatives by gate and up.
__device__ __forceinline__ float act_one_grad(float z, float d, int act) {
  if (act == MOE_ACT_SRELU) return z <= 0.f ? 0.f : d * (2.f * z);
  if (act == MOE_ACT_GELU) return d * gelu_grad(z).x;
  if (act == MOE_ACT_SILU) {
    const float s = sigmoidf_(z);
    return d * (s + z * s * (1.f - s));
  }
  return d;
}
__device__ __forceinline__ float2 act_two_grad(float g, float u, float d, const ActParams& p) {
  if (p.act == MOE_ACT_SWIGLU) {
    const float s = sigmoidf_(g);
    return make_float2(d * ((s + g * s * (1.f - s)) * u), d * (g * s));
  }
  if (p.act == MOE_ACT_GEGLU) {
    const float2 f = gelu_grad(g);
    return make_float2(d * (f.x * u), d * f.y);
  }
  const float gc = clamp_(g, p.limit), uc = clamp_(u, p.limit), s = sigmoidf_(p.alpha * gc), gs = gc * s;
  // inclusive, as the layer's; a NaN counts as inside
  const bool gin = !(fabsf(g) > p.limit), uin = !(fabsf(u) > p.limit);
  return make_float2(gin ? d * ((s + p.alpha * gs * (1.f - s)) * uc) : 0.f, uin ? d * gs : 0.f);
}

struct LinearArgs {
  int R, N, K;                  // N: output columns; weight rows: N, gated 2 N
  ActParams act;
  int dtype, wdtype;            // wdtype: of bias and db
  const void* x; int64_t ldx;
  const void* w; int64_t ldw;
  const void* bias;             // nullable
  const void* res; int64_t ldr; // nullable; may be out
  void* z; int64_t ldz;         // forward: nullable output; backward: input
  void* out; int64_t ldo;
  const void* dout; int64_t lddout;
  void* dz; int64_t lddz;
  void* dx; int64_t lddx;
  void* dw; int64_t lddw;
  void* db;
  int32_t* status;
  float* part;
};
int64_t linear_part_bytes(int R, int rows, int K, bool backward);
cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t st);
cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t st);

// ---- the layer for a few tokens (layer16.cu) -------------------------------------
struct Layer16Args {
  int T, H, I, E, k, S;         // S: shared experts
  ActParams act;
  float rs;
  int dtype;
  const void* x; int64_t ldx;
  const float* W_r;             // router weights, or
  const float* logits;          // logits, or neither: ids and w are inputs
  const void* w1; int64_t g1, ld1;
  const float* b1;              // nullable
  const void* w2; int64_t g2, ld2;
  void* out; int64_t ldo;
  int32_t* ids; float* w;
  uint8_t* ws;                  // past the status word's block; scratch
  int32_t* status;
  int32_t* arrive;              // [kL16Arrive] zero between calls: next to the status word, where no operator
                                // that shares the workspace writes
};
constexpr int kL16Arrive = 8;
int64_t layer16_ws_bytes(int T, int H, int I, int E, int k, int S);
cudaError_t launch_layer16(const Layer16Args& a, cudaStream_t st);

}  // namespace moe
