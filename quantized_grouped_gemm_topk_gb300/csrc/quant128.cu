// Quantisers of the FP8 128-block product: E4M3 codes with one fp32 scale for
// 1 x 128 elements of a row (activations, gradients) or for 128 x 128 of a
// weight matrix, the latter with a transposed copy on request (the same codes
// and scales, for the product with the transposed weight).
//
//   s = max(amax fl(1/448), 2^-126),  q = E4M3(v fl(1/s)), nearest, ties to even
//
// amax is over the block's finite values: an infinity or NaN becomes a NaN
// code and leaves the others as they are. Columns and rows past the matrix
// count as zeros and are not written.
// Bound: HBM (3 bytes an element, 4 with the transposed copy), one pass: a
// half-warp holds a row's block in registers; a CTA a 128 x 128 block, whose
// codes cross shared memory once for the transposed copy.
#include "ops.cuh"

namespace moe {

constexpr int kQThreads = 256;

// Eight consecutive elements c .. c + 7 of a row of n (zeros from n on). VEC:
// 16-byte aligned; otherwise rows at any alignment.
template <typename E, bool VEC>
__device__ __forceinline__ void load_run8(float (&v)[8], const typename E::raw* p, int c, int n) {
  constexpr int kES = (int)sizeof(typename E::raw), kPer = 16 / kES;
#pragma unroll
  for (int k = 0; k < 8 / kPer; ++k) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if constexpr (VEC) {
      if (c + k * kPer < n) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + c + k * kPer);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      }
    } else {
      load_any<kES, 16>(w, p + c + k * kPer, p, p + n);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (kES == 2) v[k * kPer + j] = E::to((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
      else v[k * kPer + j] = __uint_as_float(w[j]);
    }
  }
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = f32x2_to_e4m3x2(code_arg(v[2 * j], inv), code_arg(v[2 * j + 1], inv));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ float mag8(const float (&v)[8]) {
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, finite_mag(v[j]));
  return am;
}
template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* p, uint2 w, int c, int n) {
  if (c >= n) return;
  if constexpr (VEC) *reinterpret_cast<uint2*>(p + c) = w;
  else store_bytes8(p + c, w, n - c);
}

template <typename E, bool VEC>
__global__ void __launch_bounds__(kQThreads) k_quant128_rows(QuantRowsArgs a) {
  pdl_enter();
  const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int nb = (a.C + kQBlock - 1) / kQBlock;
  const int64_t items = a.R * nb, step = (int64_t)gridDim.x * (kQThreads / 16);
  for (int64_t it0 = (int64_t)blockIdx.x * (kQThreads / 16) + (hw & ~1); it0 < items; it0 += step) {
    const int64_t it = it0 + (hw & 1);
    const bool live = it < items;
    const int64_t row = live ? it / nb : 0;
    const int b = live ? (int)(it - row * nb) : 0;
    float v[8];
    const int c = b * kQBlock + l * 8;
    load_run8<E, VEC>(v, reinterpret_cast<const typename E::raw*>(a.x) + row * a.ldx, c, live ? a.C : 0);
    float am = mag8(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
    const float s = block_scale(am);
    if (live) store_codes8<VEC>(a.q + row * a.ldq, codes8(v, 1.0f / s), c, a.C);
    if (live && l == 0) a.s[row * a.lds + b] = s;
  }
}

// One CTA per 128 x 128 block of a group: thread (y, x) = (id / 16, id % 16)
// holds columns 8x .. 8x + 7 of rows y, y + 16, ...
template <typename E, bool VEC>
__global__ void __launch_bounds__(kQThreads) k_quant128_weights(QuantWeightsArgs a) {
  pdl_enter();
  __shared__ float red[kQThreads / 32];
  // codes of the block, column-major, 4-byte words of four rows; the row of
  // words is padded by one so a column's writes spread over the banks
  __shared__ uint8_t tile[kQBlock][kQBlock + 4];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int nb = (a.N + kQBlock - 1) / kQBlock, kb = (a.K + kQBlock - 1) / kQBlock;
  const int64_t blocks = (int64_t)a.G * nb * kb;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int64_t g = blk / ((int64_t)nb * kb);
    const int bi = (int)(blk - g * nb * kb), n0 = bi / kb * kQBlock, k0 = bi % kb * kQBlock;
    const int nn = min(kQBlock, a.N - n0), kn = min(kQBlock, a.K - k0);
    const typename E::raw* w = reinterpret_cast<const typename E::raw*>(a.w) + g * a.wg + (int64_t)n0 * a.ldw;
    float v[8][8];
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = y + 16 * i;
      load_run8<E, VEC>(v[i], w + (int64_t)min(r, nn - 1) * a.ldw, k0 + x * 8, r < nn ? a.K : 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) am = fmaxf(am, mag8(v[i]));
    am = warp_max(am);
    __syncthreads();               // the last block's reads of red and tile are done
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = am;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQThreads / 32; ++i) am = fmaxf(am, red[i]);
    const float s = block_scale(am), inv = 1.0f / s;
    uint8_t* q = a.q + g * a.qg + (int64_t)n0 * a.ldq + k0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = y + 16 * i;
      const uint2 c = codes8(v[i], inv);
      if (r < nn) store_codes8<VEC>(q + (int64_t)r * a.ldq, c, x * 8, kn);
      if (a.qt) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[x * 8 + j][r] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
      }
    }
    if (threadIdx.x == 0) {
      a.s[(g * nb + n0 / kQBlock) * kb + k0 / kQBlock] = s;
      if (a.qt) a.st[(g * kb + k0 / kQBlock) * nb + n0 / kQBlock] = s;
    }
    if (a.qt) {
      __syncthreads();
      // transposed rows (one per column k of the block), four codes a lane
      uint8_t* qt = a.qt + g * a.qtg + (int64_t)k0 * a.ldqt + n0;
      const int c4 = (threadIdx.x & 31) * 4;
      for (int r = threadIdx.x >> 5; r < kn; r += kQThreads / 32) {
        const uint32_t wd = *reinterpret_cast<const uint32_t*>(&tile[r][c4]);
        uint8_t* d = qt + (int64_t)r * a.ldqt + c4;
        if (VEC && c4 + 4 <= nn) {
          *reinterpret_cast<uint32_t*>(d) = wd;
        } else {
          for (int j = 0; j < 4 && c4 + j < nn; ++j) d[j] = (uint8_t)(wd >> (8 * j));
        }
      }
    }
  }
}

// ---- host ----------------------------------------------------------------------
static bool al(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename E>
static cudaError_t rows_t(const QuantRowsArgs& a, cudaStream_t st) {
  const int per = 16 / (int)sizeof(typename E::raw);
  const bool vec = a.C % 8 == 0 && a.ldx % per == 0 && a.ldq % 8 == 0 && al(a.x, 16) && al(a.q, 8);
  const int64_t items = a.R * ((a.C + kQBlock - 1) / kQBlock);
  const int64_t g = std::min<int64_t>((items + kQThreads / 16 - 1) / (kQThreads / 16), (int64_t)device_sms() * 32);
  note_launch();
  if (vec) return launch_pdl(k_quant128_rows<E, true>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
  return launch_pdl(k_quant128_rows<E, false>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
}
template <typename E>
static cudaError_t weights_t(const QuantWeightsArgs& a, cudaStream_t st) {
  const int per = 16 / (int)sizeof(typename E::raw);
  const bool vec = a.K % 8 == 0 && a.ldw % per == 0 && a.wg % per == 0 && a.ldq % 8 == 0 && a.qg % 8 == 0 &&
                   al(a.w, 16) && al(a.q, 8) && (!a.qt || (a.ldqt % 4 == 0 && a.qtg % 4 == 0 && al(a.qt, 4)));
  const int64_t blocks = (int64_t)a.G * ((a.N + kQBlock - 1) / kQBlock) * ((a.K + kQBlock - 1) / kQBlock);
  const int64_t g = std::min<int64_t>(blocks, (int64_t)device_sms() * 16);
  note_launch();
  if (vec) return launch_pdl(k_quant128_weights<E, true>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
  return launch_pdl(k_quant128_weights<E, false>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
}

cudaError_t launch_quant128_rows(const QuantRowsArgs& a, cudaStream_t st) {
  if (a.dtype == MOE_DT_F32) return rows_t<F32>(a, st);
  return a.dtype == MOE_DT_F16 ? rows_t<F16>(a, st) : rows_t<Bf16>(a, st);
}
cudaError_t launch_quant128_weights(const QuantWeightsArgs& a, cudaStream_t st) {
  if (a.dtype == MOE_DT_F32) return weights_t<F32>(a, st);
  return a.dtype == MOE_DT_F16 ? weights_t<F16>(a, st) : weights_t<Bf16>(a, st);
}

}  // namespace moe
