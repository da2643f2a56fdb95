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

// V consecutive elements as one access (V * sizeof(raw) is 16, or V is 1).
template <typename E, int V>
struct Pack {
  typename E::raw v[V];
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
// Column tile and pieces of the reduction, from the sizes alone.
struct MmPlan {
  int bn, S;
};
MmPlan mm_plan(int kind, int R, int N, int K, int G);
int mm_splits(int kind, int R, int N, int K, int G);
// Adds the partial sums of a split product into out.
cudaError_t launch_mm_join(const MmArgs& a, bool wgrad, cudaStream_t st);
// Tensor map of rank dimensions (innermost first; strides in elements, from
// the second axis on), 128-byte swizzle, zeros past every edge.
bool make_tmap(CUtensorMap* map, const void* base, int esize, int rank, const int64_t* dims, const int64_t* strides,
               const int* box);
cudaError_t launch_mm16(const MmArgs& a, bool wgrad, cudaStream_t st);
cudaError_t launch_mm_fp8(const MmArgs& a, cudaStream_t st);

}  // namespace moe
