// Dense products with bias, activation and residual in the epilogue:
//
//   z = x w^T + b, out = act(z) + residual
//
// and their backward from the saved z: dz = dout act'(z), dx = dz w, dw = dz^T x,
// db = the column sums of dz.
//
// Forward, many rows: tcgen05 on pairs of SMs (cta_group::2), tiles of 256 rows of
// x (the MMA's M, a lane of tensor memory each) by up to 256 columns. Rows on the
// M side, unlike the grouped products: a thread then holds neighbouring columns of
// one row, and of a gated tile (as many gate as up columns: the first CTA of the
// pair copies the gate's weights, the second the up's) both halves of each of its
// outputs, so the activation needs no exchange. Few rows: few16.cu.
#include "few16.cuh"
#include "tc.cuh"

namespace moe {

// ---- forward, many rows -------------------------------------------------------------
constexpr int kLH = 64;               // reduction of a half stage: one 128-byte swizzle row
constexpr int kLK = 2 * kLH;          // of a stage: two halves behind one barrier, freed one by one
constexpr int kLM = 128;              // rows of x a CTA
constexpr int kLStages = 3;
constexpr int kLThreads = 384;
constexpr int kLA = kLM * kLH * 2;    // bytes of a half of x's rows
constexpr int kLB = kLM * kLH * 2;    // and of the weights', at most
constexpr int kLRow = 80;             // bytes of a row of a warp's 32 x 32 staging block
constexpr int kLWarp = 32 * kLRow;
constexpr int kLSmem = 1024 + 1024 + 8 * kLWarp + kLStages * 2 * (kLA + kLB);

struct LinMaps {
  CUtensorMap x, w;
};
struct LinArgs {
  LinearArgs a;
  int bn;               // columns of an MMA: the tile's, gated twice those
  int mt, nt;           // tiles of rows and of columns
  int group;            // tiles of rows that follow each other before the next column tile
};

// The u-th tile: `group` row tiles by column tile by column tile, so that the pairs
// that run at a time share both operands' panels in L2.
__device__ __forceinline__ void lin_tile(const LinArgs& g, int u, int& m, int& n) {
  const int blk = u / (g.group * g.nt), left = min(g.group, g.mt - blk * g.group), v = u - blk * g.group * g.nt;
  n = v / left;
  m = blk * g.group + v - n * left;
}

// A warp's block of nr x nc <= 32 x 32 elements at p (row stride ld), by way of its
// staging memory, between rows of the block held by lanes and whole segments of
// memory; vec: rows start on 16 bytes.
__device__ __forceinline__ void block_in(uint8_t* st, const uint16_t* p, int64_t ld, int nr, int nc, int lane) {
  // at any alignment, an element a lane; many rows in flight
#pragma unroll
  for (int r = 0; r < 32; r += 16) {
    uint16_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = r + i < nr && lane < nc ? p[(r + i) * ld + lane] : (uint16_t)0;
#pragma unroll
    for (int i = 0; i < 16; ++i) *reinterpret_cast<uint16_t*>(st + (r + i) * kLRow + 2 * lane) = v[i];
  }
}
// y += the lane's row of the block in staging memory.
template <typename E>
__device__ __forceinline__ void add_row(uint8_t* st, int lane, float (&y)[32]) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(st + lane * kLRow + 16 * i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[8 * i + 2 * j] += E::to((uint16_t)(w[j] & 0xffffu));
      y[8 * i + 2 * j + 1] += E::to((uint16_t)(w[j] >> 16));
    }
  }
  __syncwarp();
}
template <typename E>
__device__ __forceinline__ void block_out(uint8_t* st, uint16_t* p, int64_t ld, int nr, int nc, bool vec, int lane, const float (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(st + lane * kLRow + 16 * i) =
        make_uint4(E::from2(r[8 * i], r[8 * i + 1]), E::from2(r[8 * i + 2], r[8 * i + 3]), E::from2(r[8 * i + 4], r[8 * i + 5]),
                   E::from2(r[8 * i + 6], r[8 * i + 7]));
  __syncwarp();
  if (vec && nc >= 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (lane >> 2) + 8 * i, part = lane & 3;
      if (row < nr) *reinterpret_cast<uint4*>(p + row * ld + 8 * part) = *reinterpret_cast<const uint4*>(st + row * kLRow + 16 * part);
    }
  } else {
#pragma unroll 8
    for (int row = 0; row < 32; ++row)
      if (row < nr && lane < nc) p[row * ld + lane] = *reinterpret_cast<const uint16_t*>(st + row * kLRow + 2 * lane);
  }
  __syncwarp();
}
__device__ __forceinline__ bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

template <typename E, bool GATED>
__global__ void __launch_bounds__(kLThreads, 1) k_linear(const LinArgs g, const __grid_constant__ LinMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* empty = full + kLStages;            // of each half
  uint64_t* accfull = empty + 2 * kLStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* ring = base + 1024;                  // [stage][half][x, w]
  uint8_t* staging = ring + kLStages * 2 * (kLA + kLB);
  const LinearArgs& a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)tc::cluster_rank();
  const int first = blockIdx.x / 2, stride = gridDim.x / 2, U = g.mt * g.nt;
  const int fn = GATED ? g.bn / 2 : g.bn;       // columns of out a tile
  const int nk = (a.K + kLK - 1) / kLK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kLStages; ++i) {
      tc::mbar_init(&full[i], 2);               // the first CTA's two copying warps, which expect both CTAs' bytes
      tc::mbar_init(&empty[2 * i], 1);
      tc::mbar_init(&empty[2 * i + 1], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], 1);
      tc::mbar_init(&accempty[i], 16);          // the epilogue warps of both CTAs
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.x);
    tc::prefetch_tmap(&maps.w);
  }
  if (warp == 1) tc::tmem_alloc_pair(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                           // the peer's barriers are initialised before anything reaches them
  tc::fence_after_sync();
  pdl_enter();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_u = tc::smem_u32(full), empty_u = tc::smem_u32(empty), ring_u = tc::smem_u32(ring);

  if (warp == 0 || warp == 2) {
    // ---------------- copies: warp 0 x, warp 2 w ----------------
    if (lane == 0) {
      const bool isw = warp == 2;
      const uint32_t lead = tc::peer_smem(full, 0), bytes = isw ? g.bn / 2 * kLH * 2 : kLA;
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true;
      for (int u = first; ok && u < U; u += stride) {
        int tm, tn;
        lin_tile(g, u, tm, tn);
        // a CTA's rows of x; its half of the MMA's columns, gated: gate or up
        const int row = isw ? tn * fn + (GATED ? 0 : rank * (g.bn / 2)) : tm * 2 * kLM + rank * kLM;
        for (int kb = 0; ok && kb < nk; ++kb) {
          const int k = kb * kLK, halves = a.K - k > kLH ? 2 : 1;
          for (int s = 0; s < 2; ++s) {
            if (!tc::bar_wait(empty_u + 16 * slot + 8 * s, phase, abort)) { ok = false; break; }
            if (s == 0 && rank == 0) tc::bar_arrive_expect_tx(full_u + 8 * slot, 2 * bytes * halves);
            if (s == halves) break;
            const uint32_t dst = ring_u + (2 * slot + s) * (kLA + kLB) + (isw ? kLA : 0);
            if (isw) tc::tma_load_3d_pair(dst, &maps.w, k + s * kLH, row, GATED ? rank : 0, lead + 8 * slot);
            else tc::tma_load_2d_pair(dst, &maps.x, k + s * kLH, row, lead + 8 * slot);
            if (s == 0) ++issued;
          }
          if (ok && ++slot == kLStages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok || *abort) {
        // wind-down: the copies in flight (the second CTA's report elsewhere, and the other
        // warp may have stopped earlier: the limit ends those waits)
        volatile int never = 0;
        const uint32_t n = issued < kLStages ? issued : kLStages;
        for (uint32_t i = 0; i < n; ++i) {
          const uint32_t i2 = issued - 1 - i;
          tc::mbar_wait(&full[i2 % kLStages], (i2 / kLStages) & 1, &never, 100000000ll);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    if (lane == 0 && rank == 0) {
      const uint64_t d0 = tc::smem_desc_sw128(ring_u);
      const uint32_t hi = (uint32_t)(d0 >> 32), step = (kLA + kLB) / 16;
      const uint32_t idesc = tc::idesc_16bit(2 * kLM, g.bn, a.dtype == MOE_DT_BF16, 0, 0);
      uint32_t ad = (uint32_t)d0, phase = 0, count = 0;
      int slot = 0;
      bool ok = true, ready = false;        // ready: the next stage is known to have landed
      for (int u = first; ok && u < U; u += stride, ++count) {
        const int d = count & 1;
        if (!tc::mbar_wait(&accempty[d], ((count >> 1) & 1) ^ 1, abort)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t dt = tmem + d * 256;
        uint32_t acc = 0;
        for (int left = a.K; left > 0; left -= kLK) {
          if (!ready && !tc::bar_wait(full_u + 8 * slot, phase, abort)) { ok = false; break; }
          const uint32_t done = empty_u + 16 * slot, now = ad;
          ad += 2 * step;
          if (++slot == kLStages) {
            slot = 0;
            phase ^= 1;
            ad = (uint32_t)d0;
          }
          // asked now, so that the answer's latency passes behind the MMAs' issue
          ready = tc::bar_test(full_u + 8 * slot, phase);
          tc::fence_after_sync();
          tc::mma_f16_x4<2>(dt, now, hi, 2, now + kLA / 16, hi, 2, idesc, acc);
          tc::bar_commit_pair(done);
          acc = 1;
          if (left > kLH) tc::mma_f16_x4<2>(dt, now + step, hi, 2, now + step + kLA / 16, hi, 2, idesc, 1u);
          tc::bar_commit_pair(done + 8);
        }
        if (ok) tc::mma_commit_pair(&accfull[d]);
      }
      // every MMA of this thread has completed once `drain` fires
      tc::mma_commit_pair(drain);
      volatile int never = 0;
      tc::mbar_wait(drain, 0, &never, 400000000ll);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    // All eight warps take each tile, 32 columns by 32 columns: four of them a lane
    // of tensor memory each, the other four the next 32. What a block reads from
    // memory (biases, the residual) is asked for ahead.
    const int wg = (warp - 4) >> 2, q = warp & 3;
    uint8_t* st = staging + (warp - 4) * kLWarp;
    const uint16_t* res = reinterpret_cast<const uint16_t*>(a.res);
    uint16_t *z = reinterpret_cast<uint16_t*>(a.z), *out = reinterpret_cast<uint16_t*>(a.out);
    const bool vo = rows16(out, a.ldo), vr = rows16(res, a.ldr), vz = rows16(z, a.ldz), vu = vz && a.N % 8 == 0;
    auto bias = [&](int64_t f) {
      return a.wdtype == MOE_DT_F32 ? reinterpret_cast<const float*>(a.bias)[f] : E::to(reinterpret_cast<const uint16_t*>(a.bias)[f]);
    };
    constexpr int kBlocks = GATED ? 2 : 4;      // of 32 columns, that a warp takes of a tile at most
    uint32_t count = 0;
    for (int u = first; u < U; u += stride, ++count) {
      int tm, tn;
      lin_tile(g, u, tm, tn);
      const int d = count & 1;
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + d * 256;
      const int64_t r0 = (int64_t)tm * 2 * kLM + rank * kLM + q * 32;
      const int nr = (int)max((int64_t)0, min((int64_t)32, a.R - r0));
      const int cols = min(fn, a.N - tn * fn);
      float bl[kBlocks], bu[kBlocks];
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        const int c = 32 * (wg + 2 * i) + lane;
        bl[i] = a.bias && c < cols ? bias((int64_t)tn * fn + c) : 0.f;
        bu[i] = GATED && a.bias && c < cols ? bias((int64_t)a.N + (int64_t)tn * fn + c) : 0.f;
      }
      uint4 ahead[4];       // the next block's residual, as block_in holds it
      const uint16_t* rp = res ? res + r0 * a.ldr + (int64_t)tn * fn : nullptr;
      auto fetch = [&](int c) {
        if (!res || !vr || c + 32 > cols) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (lane >> 2) + 8 * i;
          if (row < nr) ahead[i] = *reinterpret_cast<const uint4*>(rp + row * a.ldr + c + 8 * (lane & 3));
        }
      };
      fetch(32 * wg);
      const bool got = tc::mbar_wait(&accfull[d], (count >> 1) & 1, abort);
      if (!__all_sync(kFull, got)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int blk = 0; blk < kBlocks; ++blk) {
        const int c = 32 * (wg + 2 * blk), nc = min(32, cols - c);
        if (nc <= 0) break;
        const int64_t n0 = (int64_t)tn * fn + c;
        uint32_t v[32], w[GATED ? 32 : 1];
        tc::tmem_ld32(acc + c, v);
        if constexpr (GATED) tc::tmem_ld32(acc + fn + c, w);
        tc::tmem_wait_ld();
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          y[i] = __uint_as_float(v[i]) + __shfl_sync(kFull, bl[blk], i);
          if constexpr (GATED) w[i] = __float_as_uint(__uint_as_float(w[i]) + __shfl_sync(kFull, bu[blk], i));
        }
        if (z) {
          block_out<E>(st, z + r0 * a.ldz + n0, a.ldz, nr, nc, vz, lane, y);
          if constexpr (GATED) block_out<E>(st, z + r0 * a.ldz + a.N + n0, a.ldz, nr, nc, vu, lane, reinterpret_cast<float(&)[32]>(w));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if constexpr (GATED) y[i] = act_two(y[i], __uint_as_float(w[i]), a.act);
          else y[i] = act_one(y[i], a.act.act);
        }
        if (res) {
          if (vr && nc == 32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(st + ((lane >> 2) + 8 * i) * kLRow + 16 * (lane & 3)) = ahead[i];
            fetch(c + 64);
          } else {
            block_in(st, res + r0 * a.ldr + n0, a.ldr, nr, nc, lane);
          }
          add_row<E>(st, lane, y);
        }
        block_out<E>(st, out + r0 * a.ldo + n0, a.ldo, nr, nc, vo, lane, y);
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (rank != 0) tc::mbar_arrive_peer(tc::peer_smem(&accempty[d], 0));
        else tc::mbar_arrive(&accempty[d]);
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  // neither CTA leaves while the other's MMAs read its memory or its arrivals are on their way
  tc::cluster_sync();
  if (threadIdx.x == 0 && *abort) set_status(a.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

static int64_t up(int64_t n, int64_t t) { return (n + t - 1) / t; }

template <typename E, bool GATED>
static cudaError_t launch_pairs(LinArgs& g, cudaStream_t st) {
  const LinearArgs& a = g.a;
  // pairs that are resident at once, asked once per device
  static std::atomic<bool> done[kMaxDevices] = {};
  static std::atomic<int> pairs[kMaxDevices] = {};
  cudaError_t e = set_smem_once((const void*)k_linear<E, GATED>, kLSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kLThreads);
  cfg.dynamicSmemBytes = kLSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const bool slot = dev >= 0 && dev < kMaxDevices;
  int np = slot ? pairs[dev].load(std::memory_order_acquire) : 0;
  if (np <= 0) {
    cfg.gridDim = dim3(2 * (device_sms() / 2));
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&np, k_linear<E, GATED>, &cfg) != cudaSuccess || np <= 0) np = std::max(1, device_sms() / 2);
    if (slot) pairs[dev].store(np, std::memory_order_release);
  }
  // columns a tile: the width whose rounds over the pairs cost least, its own
  // columns and a fixed part each
  constexpr int kStep = GATED ? 64 : 32;        // of the MMA: whole blocks of 32 columns of out
  g.mt = (int)up(a.R, 2 * kLM);
  int64_t least = INT64_MAX;
  for (int bn = 256; bn >= 64; bn -= kStep) {
    const int64_t nt = up(a.N, GATED ? bn / 2 : bn), cost = up(g.mt * nt, np) * (bn + 64);
    if (cost < least) {
      least = cost;
      g.bn = bn;
      g.nt = (int)nt;
    }
  }
  if ((int64_t)g.mt * g.nt >= (1ll << 31) - 4096) return cudaErrorInvalidValue;
  g.group = 8;
  LinMaps maps;
  const int64_t xd[2] = {a.K, a.R}, xs[1] = {a.ldx};
  const int64_t wd[3] = {a.K, a.N, GATED ? 2 : 1}, ws[2] = {a.ldw, GATED ? (int64_t)a.N * a.ldw : a.ldw};
  const int xb[2] = {kLH, kLM}, wb[3] = {kLH, g.bn / 2, 1};
  if (!make_tmap(&maps.x, a.x, 2, 2, xd, xs, xb) || !make_tmap(&maps.w, a.w, 2, 3, wd, ws, wb)) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(np, (int64_t)g.mt * g.nt));
  cfg.numAttrs = 2;
  note_launch();
  return cudaLaunchKernelEx(&cfg, k_linear<E, GATED>, g, maps);
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t st) {
  // Few rows, or too few columns for the pairs: 128 rows x 7168 x 2048 TODO
  if (a.R <= 128 || (a.R <= kFewRows && (int64_t)a.N * (act_gated(a.act.act) ? 2 : 1) < 40 * 64)) {
    FewArgs f = {};
    f.R = a.R; f.K1 = a.K; f.F1 = a.N; f.act = a.act; f.dtype = a.dtype; f.wdtype = a.wdtype; f.status = a.status;
    f.bias = a.bias; f.res = a.res; f.ldr = a.ldr; f.z = a.z; f.ldz = a.ldz; f.out = a.out; f.ldo = a.ldo;
    return launch_few_linear(f, a.x, a.ldx, a.w, a.ldw, st);
  }
  LinArgs g = {};
  g.a = a;
  const bool bf = a.dtype == MOE_DT_BF16;
  if (act_gated(a.act.act)) return bf ? launch_pairs<Bf16, true>(g, st) : launch_pairs<F16, true>(g, st);
  return bf ? launch_pairs<Bf16, false>(g, st) : launch_pairs<F16, false>(g, st);
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
