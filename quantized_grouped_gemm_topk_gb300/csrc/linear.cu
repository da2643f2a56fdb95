// Dense products with bias, activation and residual in the epilogue:
//
//   z = x w^T + b, out = act(z) + residual
//
// and their backward from the saved z: dz = dout act'(z), dx = dz w, dw = dz^T x,
// db = the column sums of dz. dz is rounded to 16 bits once, for both products (dx and
// dw are then 1.4 times as far off as their own rounding leaves them): in two parts, as
// the few tokens' layer holds its y, the products would take twice their 640 us at
// 16384 x 2 x 2880 x 2880, where the tensor cores are what bounds them.
//
// Few rows of the forward run in few16.cu, many, and the backward's products, in
// linear_pairs.cuh.
#include "linear.cuh"

namespace moe {

// ---- forward ----------------------------------------------------------------------
static cudaError_t launch_pairs(LinArgs& g, int mode, bool gated, cudaStream_t st) {
  return g.a.dtype == MOE_DT_BF16 ? launch_pairs_bf16(g, mode, gated, st) : launch_pairs_f16(g, mode, gated, st);
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t st) {
  const bool gated = act_gated(a.act.act);
  // Few rows: there a tile's weights are shared out over all SMs, and the time grows with
  // the rows; on pairs, one tile of 256 rows however many there are, with the
  // reduction (4 us and 3.8 for each 1000 of it). In us, here and on pairs: 64 rows x
  // 7168 x 2048 11.0, 13.4; 128 rows 15.1, 13.6, x 2 x 2880 x 2880 17.3, 17.4, x 2880 x
  // 7168 20.4, 30.7; 256 rows x 7168 x 2048 23.8, 13.9, x 1440 x 2880 12.8, 15.9, x 2 x
  // 1024 x 512 6.8, 6.2.
  const int64_t rows = (int64_t)a.N * (gated ? 2 : 1);
  if (a.R <= 64 || (a.R <= kFewRows && a.R * rows < 256ll * a.K)) {
    FewArgs f = {};
    f.R = a.R; f.K1 = a.K; f.F1 = a.N; f.act = a.act; f.dtype = a.dtype; f.wdtype = a.wdtype; f.status = a.status;
    f.bias = a.bias; f.res = a.res; f.ldr = a.ldr; f.z = a.z; f.ldz = a.ldz; f.out = a.out; f.ldo = a.ldo;
    return launch_few_linear(f, a.x, a.ldx, a.w, a.ldw, st);
  }
  LinArgs g = {};
  g.a = a;
  g.M = a.R; g.N = a.N; g.K = a.K; g.out = reinterpret_cast<uint16_t*>(a.out); g.ldo = a.ldo;
  return launch_pairs(g, kLinFwd, gated, st);
}

// ---- backward ---------------------------------------------------------------------
// dz = dout act'(z) and, where asked for, partial sums of its columns: a lane
// owns eight columns, a CTA's warps share out its rows. part [blocks][rows of w].
// Bound: HBM where rows start on 16 bytes (VEC): the next row's units are asked for
// before a row is worked on, and the activation is known to the compiler (with eight
// values an array and the activation chosen by element 16384 x 2880, clamped SwiGLU,
// took 119 us).
constexpr int kDzCols = 256, kDzWarps = 8;
constexpr int kDzMaxBlocks = 128;      // row blocks

// Eight elements: a 16-byte unit, or (any alignment, or the row's last) one by one.
template <bool VEC>
__device__ __forceinline__ uint4 dz_load(const uint16_t* p, int n) {
  if constexpr (VEC) {
    if (n >= 8) return *reinterpret_cast<const uint4*>(p);
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool VEC>
__device__ __forceinline__ void dz_store(uint16_t* p, const uint32_t (&w)[4], int n) {
  if (VEC && n >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

template <typename E, int ACT, bool VEC>
__global__ void __launch_bounds__(32 * kDzWarps, 3) k_linear_dz(const LinearArgs a) {
  constexpr bool GATED = act_gated(ACT), NONE = ACT == MOE_ACT_NONE;
  constexpr int HV = GATED ? 2 : 1;
  const ActParams act = {ACT, a.act.alpha, a.act.limit};
  __shared__ float red[kDzWarps][HV][kDzCols];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * kDzCols + lane * 8, n = a.N - c;
  const uint16_t *dout = reinterpret_cast<const uint16_t*>(a.dout) + c, *z = reinterpret_cast<const uint16_t*>(a.z) + c;
  uint16_t* dz = reinterpret_cast<uint16_t*>(a.dz) + c;
  float s[HV][8] = {};
  if (n > 0) {
    const int64_t r1 = (int64_t)a.R * (blockIdx.y + 1) / gridDim.y;
    int64_t r = (int64_t)a.R * blockIdx.y / gridDim.y + warp;
    uint4 d = {}, g = {}, u = {};
    auto fetch = [&](int64_t rr) {
      d = dz_load<VEC>(dout + rr * a.lddout, n);
      if (!NONE) g = dz_load<VEC>(z + rr * a.ldz, n);
      if (GATED) u = dz_load<VEC>(z + rr * a.ldz + a.N, n);
    };
    if (r < r1) fetch(r);
    for (; r < r1; r += kDzWarps) {
      const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
      if (r + kDzWarps < r1) fetch(r + kDzWarps);
      uint32_t go[4], uo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float og[2], ou[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float dv = E::to((uint16_t)(k ? dw[j] >> 16 : dw[j] & 0xffffu)), gv = E::to((uint16_t)(k ? gw[j] >> 16 : gw[j] & 0xffffu));
          if constexpr (GATED) {
            const float2 t = act_two_grad(gv, E::to((uint16_t)(k ? uw[j] >> 16 : uw[j] & 0xffffu)), dv, act);
            og[k] = t.x;
            ou[k] = t.y;
            s[HV - 1][2 * j + k] += t.y;
          } else {
            og[k] = NONE ? dv : act_one_grad(gv, dv, ACT);
          }
          s[0][2 * j + k] += og[k];
        }
        go[j] = E::from2(og[0], og[1]);
        if constexpr (GATED) uo[j] = E::from2(ou[0], ou[1]);
      }
      if constexpr (!NONE) dz_store<VEC>(dz + r * a.lddz, go, n);
      if constexpr (GATED) dz_store<VEC>(dz + r * a.lddz + a.N, uo, n);
    }
  }
  if (!a.db) return;
#pragma unroll
  for (int h = 0; h < HV; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp][h][lane * 8 + i] = s[h][i];
  __syncthreads();
  for (int i = threadIdx.x; i < HV * kDzCols; i += 32 * kDzWarps) {
    const int h = i / kDzCols, cc = i % kDzCols;
    if (blockIdx.x * kDzCols + cc >= a.N) continue;
    float v = red[0][h][cc];
#pragma unroll
    for (int w = 1; w < kDzWarps; ++w) v += red[w][h][cc];
    a.part[(int64_t)blockIdx.y * HV * a.N + (int64_t)h * a.N + blockIdx.x * kDzCols + cc] = v;
  }
}

// db = the blocks' partial sums: a warp adds every eighth of them for 32 columns, the
// eight sums are added in order.
template <typename E>
__global__ void __launch_bounds__(256) k_linear_db(const float* __restrict__ part, int P, int rows, void* db, int wdtype) {
  __shared__ float red[8][32];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t c = (int64_t)blockIdx.x * 32; c < rows; c += (int64_t)gridDim.x * 32) {
    float v = 0.f;
    if (c + lane < rows)
#pragma unroll 4
      for (int p = warp; p < P; p += 8) v += part[(int64_t)p * rows + c + lane];
    red[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c + lane < rows) {
#pragma unroll
      for (int w = 1; w < 8; ++w) v += red[w][lane];
      if (wdtype == MOE_DT_F32) reinterpret_cast<float*>(db)[c + lane] = v;
      else reinterpret_cast<uint16_t*>(db)[c + lane] = E::from(v);
    }
    __syncthreads();
  }
}

// Row blocks: a CTA of eight warps each, as many as fill the SMs a few times over.
static int dz_blocks(int R, int N) {
  const int64_t cols = (N + kDzCols - 1) / kDzCols, most = std::max<int64_t>(1, std::min<int64_t>(kDzMaxBlocks, 8 * 152 / cols));
  return (int)std::max<int64_t>(1, std::min<int64_t>((R + 2 * kDzWarps - 1) / (2 * kDzWarps), most));
}
// Most floats of partial sums of R rows or fewer, of a plain or gated activation's
// columns (of half the rows of w).
static int64_t dz_part_floats(int R, int rows) {
  return (int64_t)std::max(dz_blocks(R, rows), dz_blocks(R, (rows + 1) / 2)) * rows;
}

// The workspace's partial sums. Backward: of the column sums, then those of the
// products (one after the other).
int64_t linear_part_bytes(int R, int rows, int K, bool backward) {
  if (!backward) return 0;
  return (dz_part_floats(R, rows) + 3) / 4 * 16 + std::max(mm_part_bytes(kMmRows, R, K, rows, 1), mm_part_bytes(kMmWgrad, R, rows, K, 1));
}

template <typename E>
static cudaError_t launch_dz(const LinearArgs& a, cudaStream_t st) {
  const bool gated = act_gated(a.act.act);
  const int P = dz_blocks(a.R, a.N);
  note_launch();
  // 16-byte accesses: dz's rows always start on one, a gated act's second halves where N does
  const bool vec = rows16(a.dout, a.lddout) && (a.act.act == MOE_ACT_NONE || rows16(a.z, a.ldz)) && (!gated || a.N % 8 == 0);
  void (*kernel)(LinearArgs) = nullptr;
  switch (a.act.act) {
#define MOE_DZ(act) case act: kernel = vec ? k_linear_dz<E, act, true> : k_linear_dz<E, act, false>; break
    MOE_DZ(MOE_ACT_SWIGLU);
    MOE_DZ(MOE_ACT_SWIGLU_CLAMP);
    MOE_DZ(MOE_ACT_GEGLU);
    MOE_DZ(MOE_ACT_SRELU);
    MOE_DZ(MOE_ACT_GELU);
    MOE_DZ(MOE_ACT_SILU);
    MOE_DZ(MOE_ACT_NONE);
#undef MOE_DZ
    default: return cudaErrorInvalidValue;
  }
  cudaError_t e = launch_pdl(kernel,
                             dim3((a.N + kDzCols - 1) / kDzCols, P), dim3(32 * kDzWarps), 0, st, a);
  if (e != cudaSuccess || !a.db) return e;
  const int rows = gated ? 2 * a.N : a.N;
  note_launch();
  return launch_pdl(k_linear_db<E>, dim3(std::min((rows + 31) / 32, 65535)), dim3(256), 0, st, (const float*)a.part, P, rows,
                    a.db, a.wdtype);
}

cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t st) {
  const bool plain = a.act.act == MOE_ACT_NONE;
  const int rows = act_gated(a.act.act) ? 2 * a.N : a.N;
  cudaError_t e = cudaSuccess;
  if (!plain || a.db) e = a.dtype == MOE_DT_BF16 ? launch_dz<Bf16>(a, st) : launch_dz<F16>(a, st);
  if (e != cudaSuccess) return e;
  // The products run on pairs of SMs. A long reduction of few tiles takes them long (as
  // the forward's few rows), and goes to the grouped products' kernel with one group, which
  // splits it. In us, there and on pairs: dx of 16 x 2880 x 2880 9.7, 13.5, of 200 x 4096
  // x 1024 13.7, 18.1, of 512 x 2880 x 2880 17.3, 14.6; dw of 4096 x 300 x 200 11.1, 17.6, of
  // 8192 x 128 x 4096 30, 36, of 1003 x 1441 x 1999 15.8, 10.3.
  auto split = [](int64_t M, int64_t N, int64_t red) { return red >= 2048 && up(M, 256) * up(N, 128) < 40; };
  LinArgs g = {};
  g.a = a;
  if (plain) {
    g.a.dz = const_cast<void*>(a.dout);
    g.a.lddz = a.lddout;
  }
  MmArgs m = {};
  m.R = a.R; m.G = 1; m.dtype = m.out_dtype = a.dtype; m.status = a.status;
  m.a = plain ? a.dout : a.dz;
  m.lda = plain ? a.lddout : a.lddz;
  m.part = a.part + (dz_part_floats(a.R, rows) + 3) / 4 * 4;
  if (a.dx) {
    if (!split(a.R, a.K, rows)) {
      g.M = a.R; g.N = a.K; g.K = rows; g.out = reinterpret_cast<uint16_t*>(a.dx); g.ldo = a.lddx;
      e = launch_pairs(g, kLinDx, false, st);
    } else {
      m.N = a.K; m.K = rows; m.b = a.w; m.ldb = a.ldw; m.trans_b = 1; m.out = a.dx; m.ldo = a.lddx;
      m.S = mm_splits(kMmRows, a.R, a.K, rows, 1);
      e = launch_mm16(m, false, st);
    }
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    if (!split(rows, a.K, a.R)) {
      g.M = rows; g.N = a.K; g.K = a.R; g.out = reinterpret_cast<uint16_t*>(a.dw); g.ldo = a.lddw;
      return launch_pairs(g, kLinDw, false, st);
    }
    m.N = rows; m.K = a.K; m.b = a.x; m.ldb = a.ldx; m.trans_b = 0; m.out = a.dw; m.ldo = a.lddw; m.og = 0;
    m.S = mm_splits(kMmWgrad, a.R, rows, a.K, 1);
    return launch_mm16(m, true, st);
  }
  return cudaSuccess;
}

}  // namespace moe
