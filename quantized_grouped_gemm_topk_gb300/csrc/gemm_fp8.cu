// FP8 products with a scale for each block of 128: the plain CUDA-core form (64 x 64 output tiles, 16 of the reduction at a time
// in shared memory, fp32 sums).
#include "groups.cuh"

namespace moe {

constexpr int kTile = 64, kDepth = 16, kThr = 256;

template <int KIND>
__device__ __forceinline__ float mm_a(const MmArgs& a, int64_t r, int64_t i) {
  if constexpr (KIND == kMmFp8)
    return e4m3_to_f32(reinterpret_cast<const uint8_t*>(a.a)[r * a.lda + i]) * a.sa[r * a.ldsa + i / kQBlock];
  const uint16_t v = reinterpret_cast<const uint16_t*>(a.a)[r * a.lda + i];
  return a.dtype == MOE_DT_F16 ? F16::to(v) : Bf16::to(v);
}

template <int KIND>
__global__ void __launch_bounds__(kThr) k_mm_simple(MmArgs a) {
  pdl_enter();
  __shared__ int32_t off[kMmMaxGroups + 1], uoff[kMmMaxGroups + 1];
  __shared__ int tmp[2 * kThr / 32];
  __shared__ float As[kDepth][kTile + 1], Bs[kDepth][kTile + 1];
  const bool wg = KIND == kMmWgrad;
  // rows mode: M = rows of the group, N columns, reduction K; wgrad: M = N features, columns K, reduction rows
  const int cols = wg ? a.K : a.N;
  const int nt = (cols + kTile - 1) / kTile;
  build_groups<kThr>(a.offsets, a.G, a.R, off, uoff, tmp, a.status,
                     [&](int c) { return wg ? (a.N + kTile - 1) / kTile : (c + kTile - 1) / kTile; });
  const int64_t units = (int64_t)uoff[a.G] * nt;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int ui = (int)(u / nt), n0 = (int)(u - (int64_t)ui * nt) * kTile;
    const int e = group_of_unit(uoff, a.G, ui);
    const int m0 = (ui - uoff[e]) * kTile, r0 = off[e], cnt = off[e + 1] - r0;
    const int M = wg ? a.N : cnt, red = wg ? cnt : a.K;
    const uint16_t* b16 = reinterpret_cast<const uint16_t*>(a.b);
    float acc[4][4] = {};
    for (int k0 = 0; k0 < red; k0 += kDepth) {
      for (int i = threadIdx.x; i < kTile * kDepth; i += kThr) {
        const int m = i / kDepth, k = i % kDepth, mm = m0 + m, nn = n0 + m, kk = k0 + k;
        float va = 0.f, vb = 0.f;
        if (mm < M && kk < red) va = wg ? mm_a<KIND>(a, r0 + kk, mm) : mm_a<KIND>(a, r0 + mm, kk);
        if (nn < cols && kk < red) {
          if constexpr (KIND == kMmFp8) {
            const int nb = (a.N + kQBlock - 1) / kQBlock, kb = (a.K + kQBlock - 1) / kQBlock;
            vb = e4m3_to_f32(reinterpret_cast<const uint8_t*>(a.b)[e * a.bg + nn * a.ldb + kk]) *
                 a.sb[((int64_t)e * nb + nn / kQBlock) * kb + kk / kQBlock];
          } else {
            const uint16_t v = wg ? b16[(int64_t)(r0 + kk) * a.ldb + nn]
                                  : a.trans_b ? b16[e * a.bg + (int64_t)kk * a.ldb + nn]
                                              : b16[e * a.bg + (int64_t)nn * a.ldb + kk];
            vb = a.dtype == MOE_DT_F16 ? F16::to(v) : Bf16::to(v);
          }
        }
        As[k][m] = va;
        Bs[k][m] = vb;
      }
      __syncthreads();
      for (int k = 0; k < kDepth; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty + 16 * i], Bs[k][tx + 16 * j], acc[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m >= M || n >= cols) continue;
        const int64_t at = wg ? e * a.og + (int64_t)m * a.ldo + n : (int64_t)(r0 + m) * a.ldo + n;
        if (a.out_dtype == MOE_DT_F32) reinterpret_cast<float*>(a.out)[at] = acc[i][j];
        else reinterpret_cast<uint16_t*>(a.out)[at] =
            a.out_dtype == MOE_DT_F16 ? F16::from(acc[i][j]) : Bf16::from(acc[i][j]);
      }
  }
  if (wg) return;
  // rows outside every group
  const int esize = a.out_dtype == MOE_DT_F32 ? 4 : 2;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    if (r >= off[0] && r < off[a.G]) continue;
    for (int64_t i = threadIdx.x; i < (int64_t)a.N; i += kThr) {
      if (esize == 4) reinterpret_cast<float*>(a.out)[r * a.ldo + i] = 0.f;
      else reinterpret_cast<uint16_t*>(a.out)[r * a.ldo + i] = 0;
    }
  }
}

cudaError_t launch_mm_fp8(const MmArgs& a, cudaStream_t st) {
  note_launch();
  return launch_pdl(k_mm_simple<kMmFp8>, dim3(device_sms() * 4), dim3(kThr), 0, st, a);
}

}  // namespace moe
