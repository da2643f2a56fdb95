// Dense products with bias, activation and residual in the epilogue:
//
//   z = x w^T + b, out = act(z) + residual
//
// and their backward from the saved z: dz = dout act'(z), dx = dz w, dw = dz^T x,
// db = the column sums of dz.
#include "few16.cuh"

namespace moe {

// ---- forward ----------------------------------------------------------------------
// A thread owns 4 rows x 4 columns of a 64 x 64 tile (gated: of gate and up),
// summed over K in steps of 16 through shared memory.
constexpr int kLT = 64, kLK = 16;

template <typename E, bool GATED>
__global__ void __launch_bounds__(256) k_linear_plain(const LinearArgs a) {
  constexpr int HV = GATED ? 2 : 1;
  __shared__ float xs[kLK][kLT + 1], wsm[HV][kLK][kLT + 1];
  pdl_enter();
  const uint16_t *x = reinterpret_cast<const uint16_t*>(a.x), *w = reinterpret_cast<const uint16_t*>(a.w);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kLT;
  for (int64_t r0 = (int64_t)blockIdx.y * kLT; r0 < a.R; r0 += (int64_t)gridDim.y * kLT) {
    float acc[HV][4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kLK) {
      __syncthreads();
      for (int i = threadIdx.x; i < kLT * kLK; i += 256) {
        const int r = i / kLK, c = i % kLK;
        const bool in = k0 + c < a.K;
        xs[c][r] = in && r0 + r < a.R ? E::to(x[(r0 + r) * a.ldx + k0 + c]) : 0.f;
#pragma unroll
        for (int h = 0; h < HV; ++h)
          wsm[h][c][r] = in && n0 + r < a.N ? E::to(w[((int64_t)h * a.N + n0 + r) * a.ldw + k0 + c]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kLK; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < HV; ++h)
              acc[h][i][j] = fmaf(xs[c][ty + 16 * i], wsm[h][c][tx + 16 * j], acc[h][i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (r >= a.R || n >= a.N) continue;
        float v[HV];
#pragma unroll
        for (int h = 0; h < HV; ++h) {
          v[h] = acc[h][i][j];
          const int64_t f = (int64_t)h * a.N + n;
          if (a.bias) v[h] += a.wdtype == MOE_DT_F32 ? reinterpret_cast<const float*>(a.bias)[f]
                                                     : E::to(reinterpret_cast<const uint16_t*>(a.bias)[f]);
          if (a.z) reinterpret_cast<uint16_t*>(a.z)[r * a.ldz + f] = E::from(v[h]);
        }
        float o = GATED ? act_two(v[0], v[HV - 1], a.act) : act_one(v[0], a.act.act);
        if (a.res) o += E::to(reinterpret_cast<const uint16_t*>(a.res)[r * a.ldr + n]);
        reinterpret_cast<uint16_t*>(a.out)[r * a.ldo + n] = E::from(o);
      }
  }
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t st) {
  if (a.R <= kFewRows) {
    FewArgs f = {};
    f.R = a.R; f.K1 = a.K; f.F1 = a.N; f.act = a.act; f.dtype = a.dtype; f.wdtype = a.wdtype; f.status = a.status;
    f.bias = a.bias; f.res = a.res; f.ldr = a.ldr; f.z = a.z; f.ldz = a.ldz; f.out = a.out; f.ldo = a.ldo;
    return launch_few_linear(f, a.x, a.ldx, a.w, a.ldw, st);
  }
  const dim3 grid((a.N + kLT - 1) / kLT, std::min((a.R + kLT - 1) / kLT, 65535));
  const bool bf = a.dtype == MOE_DT_BF16;
  note_launch();
  if (act_gated(a.act.act))
    return launch_pdl(bf ? k_linear_plain<Bf16, true> : k_linear_plain<F16, true>, grid, dim3(256), 0, st, a);
  return launch_pdl(bf ? k_linear_plain<Bf16, false> : k_linear_plain<F16, false>, grid, dim3(256), 0, st, a);
}

// ---- backward ---------------------------------------------------------------------
// dz = dout act'(z) and, where asked for, partial sums of its columns: a lane
// owns eight columns, a CTA's warps share out its rows. part [blocks][rows of w].
constexpr int kDzCols = 256, kDzWarps = 8;
constexpr int kDzMaxBlocks = 256;      // row blocks

template <typename E>
__device__ __forceinline__ void load8(float (&v)[8], const uint16_t* p, int n, bool vec) {
  if (vec && n >= 8) {
    Pack<E, 8> k;
    load_pack(k, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = E::to(k.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? E::to(p[i]) : 0.f;
  }
}
template <typename E>
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], int n, bool vec) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(E::from2(v[0], v[1]), E::from2(v[2], v[3]), E::from2(v[4], v[5]), E::from2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = E::from(v[i]);
  }
}
__device__ __forceinline__ bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

template <typename E, bool GATED>
__global__ void __launch_bounds__(32 * kDzWarps) k_linear_dz(const LinearArgs a) {
  constexpr int HV = GATED ? 2 : 1;
  __shared__ float red[kDzWarps][HV][kDzCols];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * kDzCols + lane * 8, n = a.N - c;
  const uint16_t *dout = reinterpret_cast<const uint16_t*>(a.dout), *z = reinterpret_cast<const uint16_t*>(a.z);
  uint16_t* dz = reinterpret_cast<uint16_t*>(a.dz);
  const bool vd = rows16(dout, a.lddout), vz = rows16(z, a.ldz) && (!GATED || a.N % 8 == 0), vo = !GATED || a.N % 8 == 0;
  float s[HV][8] = {};
  if (n > 0) {
    const int64_t r1 = (int64_t)a.R * (blockIdx.y + 1) / gridDim.y;
    for (int64_t r = (int64_t)a.R * blockIdx.y / gridDim.y + warp; r < r1; r += kDzWarps) {
      float d[8];
      load8<E>(d, dout + r * a.lddout + c, n, vd);
      if (a.act.act == MOE_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0][i] += d[i];
        continue;
      }
      float g[8], u[8];
      load8<E>(g, z + r * a.ldz + c, n, vz);
      if (GATED) load8<E>(u, z + r * a.ldz + a.N + c, n, vz);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (GATED) {
          const float2 t = act_two_grad(g[i], u[i], d[i], a.act);
          g[i] = t.x;
          u[i] = t.y;
          s[HV - 1][i] += t.y;
        } else {
          g[i] = act_one_grad(g[i], d[i], a.act.act);
        }
        s[0][i] += g[i];
      }
      store8<E>(dz + r * a.lddz + c, g, n, true);
      if (GATED) store8<E>(dz + r * a.lddz + a.N + c, u, n, vo);
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

// db = the blocks' partial sums, added in order.
template <typename E>
__global__ void __launch_bounds__(256) k_linear_db(const float* __restrict__ part, int P, int rows, void* db, int wdtype) {
  pdl_enter();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows; i += (int64_t)gridDim.x * 256) {
    float v = 0.f;
    for (int p = 0; p < P; ++p) v += part[(int64_t)p * rows + i];
    if (wdtype == MOE_DT_F32) reinterpret_cast<float*>(db)[i] = v;
    else reinterpret_cast<uint16_t*>(db)[i] = E::from(v);
  }
}

static int dz_blocks(int R) { return std::max(1, std::min((R + 4 * kDzWarps - 1) / (4 * kDzWarps), kDzMaxBlocks)); }

// The workspace's partial sums. Backward: of the column sums, then those of the
// products (one after the other).
int64_t linear_part_bytes(int R, int rows, int K, bool backward) {
  if (!backward) return 0;
  const int64_t db = (int64_t)dz_blocks(R) * rows * 4;
  return (db + 15) / 16 * 16 + std::max(mm_part_bytes(kMmRows, R, K, rows, 1), mm_part_bytes(kMmWgrad, R, rows, K, 1));
}

template <typename E>
static cudaError_t launch_dz(const LinearArgs& a, cudaStream_t st) {
  const bool gated = act_gated(a.act.act);
  const int P = dz_blocks(a.R);
  note_launch();
  cudaError_t e = launch_pdl(gated ? k_linear_dz<E, true> : k_linear_dz<E, false>,
                             dim3((a.N + kDzCols - 1) / kDzCols, P), dim3(32 * kDzWarps), 0, st, a);
  if (e != cudaSuccess || !a.db) return e;
  const int rows = gated ? 2 * a.N : a.N;
  note_launch();
  return launch_pdl(k_linear_db<E>, dim3(std::min((rows + 255) / 256, 65535)), dim3(256), 0, st, (const float*)a.part, P, rows,
                    a.db, a.wdtype);
}

cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t st) {
  const bool plain = a.act.act == MOE_ACT_NONE;
  const int rows = act_gated(a.act.act) ? 2 * a.N : a.N;
  cudaError_t e = cudaSuccess;
  if (!plain || a.db) e = a.dtype == MOE_DT_BF16 ? launch_dz<Bf16>(a, st) : launch_dz<F16>(a, st);
  if (e != cudaSuccess) return e;
  MmArgs m = {};
  m.R = a.R; m.G = 1; m.dtype = m.out_dtype = a.dtype; m.status = a.status;
  m.a = plain ? a.dout : a.dz;
  m.lda = plain ? a.lddout : a.lddz;
  m.part = a.part + ((int64_t)dz_blocks(a.R) * rows + 3) / 4 * 4;
  if (a.dx) {
    m.N = a.K; m.K = rows; m.b = a.w; m.ldb = a.ldw; m.trans_b = 1; m.out = a.dx; m.ldo = a.lddx;
    m.S = mm_splits(kMmRows, a.R, a.K, rows, 1);
    if ((e = launch_mm16(m, false, st)) != cudaSuccess) return e;
  }
  if (a.dw) {
    m.N = rows; m.K = a.K; m.b = a.x; m.ldb = a.ldx; m.trans_b = 0; m.out = a.dw; m.ldo = a.lddw; m.og = 0;
    m.S = mm_splits(kMmWgrad, a.R, rows, a.K, 1);
    return launch_mm16(m, true, st);
  }
  return cudaSuccess;
}

}  // namespace moe
