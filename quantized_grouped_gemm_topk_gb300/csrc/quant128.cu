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
// quarter-warp (fp32: a half-warp) holds a row's block in registers; a CTA a
// 128 x 128 block, whose codes cross shared memory once for the transposed
// copy.
// Measured, bf16: rows 12289 x 7168 46 us (5.7 TB/s), 8192 x 4096 19 us (5.3; 17 where
// L2 holds them), at odd alignments 8192 x 4099 30 us (3.3); weights 7168 x 4096 with the
// transposed copy 22 us (5.4), 32 x 4096 x 1024 84 us (6.4).
#include "blocks.cuh"

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

// fp32 rows: a half-warp a block, eight columns a lane.
template <bool VEC>
__global__ void __launch_bounds__(kQThreads) k_quant128_rows32(QuantRowsArgs a) {
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
    load_run8<F32, VEC>(v, reinterpret_cast<const float*>(a.x) + row * a.ldx, c, live ? a.C : 0);
    float am = mag8(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
    const float s = block_scale(am);
    if (live) store_codes8<VEC>(a.q + row * a.ldq, codes8(v, 1.0f / s), c, a.C);
    if (live && l == 0) a.s[row * a.lds + b] = s;
  }
}

// A block's scale and codes.
template <typename E>
__device__ __forceinline__ float quant_block(uint32_t (&codes)[4], const uint32_t (&w)[8], unsigned lanes) {
  uint32_t mm = mag_bits(w);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) mm = max(mm, __shfl_xor_sync(lanes, mm, o));
  float s;
  if (mm < E::kInf) {
    s = block_scale(E::to((uint16_t)mm));
    codes16<E, true>(codes, w, 1.0f / s);
  } else {
    s = finite_scale<E>(w, lanes);
    codes16<E, false>(codes, w, 1.0f / s);
  }
  return s;
}

// 16-bit rows: a quarter-warp a block, sixteen columns a lane (blocks.cuh);
// qpr quarter-warps of a CTA share a row.
template <typename E>
__global__ void __launch_bounds__(kQThreads) k_quant128_rows(QuantRowsArgs a, int qpr) {
  pdl_enter();
  const int l = threadIdx.x & 7, qw = threadIdx.x >> 3;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  const int nb = (a.C + kQBlock - 1) / kQBlock;
  const int rpc = kQThreads / 8 / qpr, rl = qw / qpr, part = qw % qpr;
  for (int64_t row = (int64_t)blockIdx.x * rpc + rl; row < a.R; row += (int64_t)gridDim.x * rpc) {
    const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + row * a.ldx;
    uint8_t* q = a.q + row * a.ldq;
    for (int b = part; b < nb; b += qpr) {
      const int c0 = b * kQBlock, n = min(kQBlock, a.C - c0);
      uint32_t w[8], codes[4];
      load16(w, x + c0, l, n);
      const float s = quant_block<E>(codes, w, lanes);
      store_codes(q + c0, codes, l, n);
      if (l == 0) a.s[row * a.lds + b] = s;
    }
  }
}

// The same for rows at any alignment: the next block's units on their way to
// shared memory during a block, the codes stored from there.
template <typename E>
__global__ void __launch_bounds__(kQThreads) k_quant128_rows_any(QuantRowsArgs a, int qpr) {
  __shared__ __align__(16) uint8_t in_smem[kQThreads / 8][2][kStageBytes];
  __shared__ __align__(16) uint8_t out_smem[kQThreads / 8][kCodeBytes];
  pdl_enter();
  const int l = threadIdx.x & 7, qw = threadIdx.x >> 3;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  const int nb = (a.C + kQBlock - 1) / kQBlock;
  const int rpc = kQThreads / 8 / qpr, rl = qw / qpr, part = qw % qpr;
  const int64_t step = (int64_t)gridDim.x * rpc;
  const uint8_t* x0 = reinterpret_cast<const uint8_t*>(a.x);
  auto fetch = [&](int64_t row, int b, int stage) {
    if (row < a.R && b < nb) fetch_block<2>(in_smem[qw][stage], x0 + row * a.ldx * 2, b * kQBlock, a.C, x0, l);
    cp_async_commit();
  };
  int stage = 0;
  int64_t row = (int64_t)blockIdx.x * rpc + rl;
  fetch(row, part, 0);
  for (; row < a.R; row += step) {
    const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + row * a.ldx;
    uint8_t* q = a.q + row * a.ldq;
    for (int b = part; b < nb; b += qpr, stage ^= 1) {
      const int c0 = b * kQBlock, n = min(kQBlock, a.C - c0);
      const bool more = b + qpr < nb;
      fetch(more ? row : row + step, more ? b + qpr : part, stage ^ 1);
      cp_async_wait<1>();
      __syncwarp(lanes);
      uint32_t w[8], codes[4];
      read16(w, in_smem[qw][stage], (int)((uintptr_t)(x + c0) & 15), l);
      const float s = quant_block<E>(codes, w, lanes);
      stage_codes(out_smem[qw], codes, l);
      __syncwarp(lanes);
      store_staged_codes(q + c0, out_smem[qw], l, n);
      __syncwarp(lanes);
      if (l == 0) a.s[row * a.lds + b] = s;
    }
  }
  cp_async_wait<0>();
}

// Bytes (i, j) of eight rows of eight -> the same transposed: row words r[i][2]
// become column words c[j][2]. Four 4 x 4 blocks by byte permutes.
__device__ __forceinline__ void transpose8x8(uint32_t (&c)[8][2], const uint2 (&r)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)       // rows 4 h .. 4 h + 3 -> word h of the columns
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // columns 4 k .. 4 k + 3
      const uint32_t a = k ? r[4 * h].y : r[4 * h].x, b = k ? r[4 * h + 1].y : r[4 * h + 1].x;
      const uint32_t d = k ? r[4 * h + 2].y : r[4 * h + 2].x, e = k ? r[4 * h + 3].y : r[4 * h + 3].x;
      const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
      const uint32_t de0 = __byte_perm(d, e, 0x5140), de1 = __byte_perm(d, e, 0x7362);
      c[4 * k][h] = __byte_perm(ab0, de0, 0x5410);
      c[4 * k + 1][h] = __byte_perm(ab0, de0, 0x7632);
      c[4 * k + 2][h] = __byte_perm(ab1, de1, 0x5410);
      c[4 * k + 3][h] = __byte_perm(ab1, de1, 0x7632);
    }
}

// One CTA per 128 x 128 block of a group: thread (y, x) = (id / 16, id % 16)
// holds columns 8x .. 8x + 7 of rows 8y .. 8y + 7. For the transposed copy
// each thread transposes its 8 x 8 codes in registers; they cross shared
// memory as 8-byte words (column, y), at y ^ x so that neither side meets a
// bank twice.
template <typename E, bool VEC>
__global__ void __launch_bounds__(kQThreads) k_quant128_weights(QuantWeightsArgs a) {
  constexpr bool k16 = sizeof(typename E::raw) == 2;
  pdl_enter();
  __shared__ float red[kQThreads / 32];
  __shared__ uint2 tile[kQBlock][16];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int nb = (a.N + kQBlock - 1) / kQBlock, kb = (a.K + kQBlock - 1) / kQBlock;
  const int64_t blocks = (int64_t)a.G * nb * kb;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int64_t g = blk / ((int64_t)nb * kb);
    const int bi = (int)(blk - g * nb * kb), n0 = bi / kb * kQBlock, k0 = bi % kb * kQBlock;
    const int nn = min(kQBlock, a.N - n0), kn = min(kQBlock, a.K - k0);
    const typename E::raw* w = reinterpret_cast<const typename E::raw*>(a.w) + g * a.wg + (int64_t)n0 * a.ldw;
    uint32_t h[k16 ? 8 : 1][4];         // 16-bit elements as they came
    float v[k16 ? 1 : 8][8];
    float am = 0.f;
    if constexpr (k16) {
      uint32_t mm = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * y + i;
        const uint16_t* p = reinterpret_cast<const uint16_t*>(w) + (int64_t)min(r, nn - 1) * a.ldw;
        const int c = k0 + x * 8, end = r < nn ? a.K : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = 0u;
        if constexpr (VEC) {
          if (c < end) {
            const uint4 u = *reinterpret_cast<const uint4*>(p + c);
            h[i][0] = u.x; h[i][1] = u.y; h[i][2] = u.z; h[i][3] = u.w;
          }
        } else {
          load_any<2, 16>(h[i], p + c, p, p + end);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mm = __vmaxu2(mm, h[i][j] & 0x7fff7fffu);
      mm = max(mm & 0xffffu, mm >> 16);
      am = E::to((uint16_t)mm);
      if (mm >= E::kInf) {              // an infinity or NaN: the largest of the finite ones
        am = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = pair_of<E>(h[i][j]);
            am = fmaxf(am, fmaxf(finite_mag(f.x), finite_mag(f.y)));
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * y + i;
        load_run8<E, VEC>(v[i], w + (int64_t)min(r, nn - 1) * a.ldw, k0 + x * 8, r < nn ? a.K : 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) am = fmaxf(am, mag8(v[i]));
    }
    am = warp_max(am);
    __syncthreads();               // the last block's reads of red and tile are done
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = am;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQThreads / 32; ++i) am = fmaxf(am, red[i]);
    const float s = block_scale(am), inv = 1.0f / s;
    uint8_t* q = a.q + g * a.qg + (int64_t)n0 * a.ldq + k0;
    uint2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (k16) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = pair_of<E>(h[i][j]);
          f[2 * j] = p.x;
          f[2 * j + 1] = p.y;
        }
        c[i] = codes8(f, inv);
      } else {
        c[i] = codes8(v[i], inv);
      }
      const int r = 8 * y + i;
      if (r < nn) store_codes8<VEC>(q + (int64_t)r * a.ldq, c[i], x * 8, kn);
    }
    if (threadIdx.x == 0) {
      a.s[(g * nb + n0 / kQBlock) * kb + k0 / kQBlock] = s;
      if (a.qt) a.st[(g * kb + k0 / kQBlock) * nb + n0 / kQBlock] = s;
    }
    if (a.qt) {
      uint32_t t[8][2];
      transpose8x8(t, c);
#pragma unroll
      for (int j = 0; j < 8; ++j) tile[8 * x + j][y ^ x] = make_uint2(t[j][0], t[j][1]);
      __syncthreads();
      // transposed rows (one per column k of the block), eight codes a lane
      uint8_t* qt = a.qt + g * a.qtg + (int64_t)k0 * a.ldqt + n0;
      for (int r = y; r < kn; r += 16) store_codes8<VEC>(qt + (int64_t)r * a.ldqt, tile[r][x ^ (r >> 3)], x * 8, nn);
    }
  }
}

// ---- host ----------------------------------------------------------------------
static bool al(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

static bool rows_vec(const QuantRowsArgs& a, int esize) {
  return a.C % 8 == 0 && a.ldx % (16 / esize) == 0 && a.ldq % 8 == 0 && al(a.x, 16) && al(a.q, 8);
}
template <typename E>
static cudaError_t rows_t(const QuantRowsArgs& a, cudaStream_t st) {
  const int qpr = quarters_a_row(a.C, kQThreads / 8), rpc = kQThreads / 8 / qpr;
  const int64_t g = std::min<int64_t>((a.R + rpc - 1) / rpc, (int64_t)device_sms() * 32);
  note_launch();
  if (rows_vec(a, 2)) return launch_pdl(k_quant128_rows<E>, dim3((unsigned)g), dim3(kQThreads), 0, st, a, qpr);
  return launch_pdl(k_quant128_rows_any<E>, dim3((unsigned)g), dim3(kQThreads), 0, st, a, qpr);
}
static cudaError_t rows_32(const QuantRowsArgs& a, cudaStream_t st) {
  const int64_t items = a.R * ((a.C + kQBlock - 1) / kQBlock);
  const int64_t g = std::min<int64_t>((items + kQThreads / 16 - 1) / (kQThreads / 16), (int64_t)device_sms() * 32);
  note_launch();
  if (rows_vec(a, 4)) return launch_pdl(k_quant128_rows32<true>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
  return launch_pdl(k_quant128_rows32<false>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
}
template <typename E>
static cudaError_t weights_t(const QuantWeightsArgs& a, cudaStream_t st) {
  const int per = 16 / (int)sizeof(typename E::raw);
  const bool vec = a.K % 8 == 0 && a.ldw % per == 0 && a.wg % per == 0 && a.ldq % 8 == 0 && a.qg % 8 == 0 &&
                   al(a.w, 16) && al(a.q, 8) && (!a.qt || (a.N % 8 == 0 && a.ldqt % 8 == 0 && a.qtg % 8 == 0 && al(a.qt, 8)));
  const int64_t blocks = (int64_t)a.G * ((a.N + kQBlock - 1) / kQBlock) * ((a.K + kQBlock - 1) / kQBlock);
  const int64_t g = std::min<int64_t>(blocks, (int64_t)device_sms() * 16);
  note_launch();
  if (vec) return launch_pdl(k_quant128_weights<E, true>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
  return launch_pdl(k_quant128_weights<E, false>, dim3((unsigned)g), dim3(kQThreads), 0, st, a);
}

cudaError_t launch_quant128_rows(const QuantRowsArgs& a, cudaStream_t st) {
  if (a.dtype == MOE_DT_F32) return rows_32(a, st);
  return a.dtype == MOE_DT_F16 ? rows_t<F16>(a, st) : rows_t<Bf16>(a, st);
}
cudaError_t launch_quant128_weights(const QuantWeightsArgs& a, cudaStream_t st) {
  if (a.dtype == MOE_DT_F32) return weights_t<F32>(a, st);
  return a.dtype == MOE_DT_F16 ? weights_t<F16>(a, st) : weights_t<Bf16>(a, st);
}

}  // namespace moe
