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
// outputs, so the activation needs no exchange. Few rows: few16.cu. The backward's
// products run in the same kernel, dw with dz's columns as M, and with the operands
// whose M or N axis is contiguous in memory (w for dx, both for dw) as they lie there.
#include "few16.cuh"
#include "tc.cuh"

namespace moe {

// ---- products of many rows ------------------------------------------------------------
constexpr int kLH = 64;               // reduction of a half stage: one 128-byte swizzle row
constexpr int kLK = 2 * kLH;          // of a stage: two halves behind one barrier, freed one by one
constexpr int kLM = 128;              // rows of x a CTA
constexpr int kLStages = 3;
constexpr int kLThreads = 384;
constexpr int kLA = kLM * kLH * 2;    // bytes of a half of x's rows
constexpr int kLB = kLM * kLH * 2;    // and of the weights', at most
constexpr int kLChunk = 64 * kLH * 2; // of 64 columns of an operand with its M / N axis contiguous
constexpr int kLRow = 80;             // bytes of a row of a warp's 32 x 32 staging block
constexpr int kLWarp = 32 * kLRow;
constexpr int kLSmem = 1024 + 1024 + 8 * kLWarp + kLStages * 2 * (kLA + kLB);

// D[M][N] of a tile: out = x w^T | dx = dz w | dw = dz^T x.
enum { kLinFwd = 0, kLinDx = 1, kLinDw = 2 };
struct LinMaps {
  CUtensorMap x, w;     // the operands A and B
};
struct LinArgs {
  LinearArgs a;
  int64_t M;            // rows of the result,
  int N, K;             // its columns (gated: of out), the reduction
  uint16_t* out; int64_t ldo;
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
__host__ __device__ __forceinline__ bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

template <typename E, int MODE, bool GATED>
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
  const int nk = (g.K + kLK - 1) / kLK;

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
      constexpr bool kMnA = MODE == kLinDw, kMnB = MODE != kLinFwd;     // M / N axis contiguous
      const int chunks = isw ? (kMnB ? (g.bn / 2 + 63) / 64 : 0) : kMnA ? kLM / 64 : 0;
      const uint32_t lead = tc::peer_smem(full, 0), bytes = chunks ? chunks * kLChunk : isw ? g.bn / 2 * kLH * 2 : kLA;
      const CUtensorMap* map = isw ? &maps.w : &maps.x;
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true;
      for (int u = first; ok && u < U; u += stride) {
        int tm, tn;
        lin_tile(g, u, tm, tn);
        // a CTA's rows of x; its half of the MMA's columns, gated: gate or up
        const int row = isw ? tn * fn + (GATED ? 0 : rank * (g.bn / 2)) : tm * 2 * kLM + rank * kLM;
        for (int kb = 0; ok && kb < nk; ++kb) {
          const int k = kb * kLK, halves = g.K - k > kLH ? 2 : 1;
          for (int s = 0; s < 2; ++s) {
            if (!tc::bar_wait(empty_u + 16 * slot + 8 * s, phase, abort)) { ok = false; break; }
            if (s == 0 && rank == 0) tc::bar_arrive_expect_tx(full_u + 8 * slot, 2 * bytes * halves);
            if (s == halves) break;
            const uint32_t dst = ring_u + (2 * slot + s) * (kLA + kLB) + (isw ? kLA : 0);
            if (isw && !kMnB) tc::tma_load_3d_pair(dst, map, k + s * kLH, row, GATED ? rank : 0, lead + 8 * slot);
            else if (!isw && !kMnA) tc::tma_load_2d_pair(dst, map, k + s * kLH, row, lead + 8 * slot);
            else
              for (int c = 0; c < chunks; ++c)
                tc::tma_load_2d_pair(dst + c * kLChunk, map, row + 64 * c, k + s * kLH, lead + 8 * slot);
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
      constexpr bool kMnA = MODE == kLinDw, kMnB = MODE != kLinFwd;
      const uint64_t ad0 = kMnA ? tc::smem_desc_mn_sw128(ring_u, kLChunk) : tc::smem_desc_sw128(ring_u);
      const uint64_t bd0 = kMnB ? tc::smem_desc_mn_sw128(ring_u + kLA, kLChunk) : tc::smem_desc_sw128(ring_u + kLA);
      // a step of K = 16: two 8-row atoms, or 32 bytes along a K-major row
      constexpr uint32_t sa = kMnA ? 2048 / 16 : 2, sb = kMnB ? 2048 / 16 : 2, step = (kLA + kLB) / 16;
      const uint32_t ahi = (uint32_t)(ad0 >> 32), bhi = (uint32_t)(bd0 >> 32), b_off = (uint32_t)bd0 - (uint32_t)ad0;
      const uint32_t idesc = tc::idesc_16bit(2 * kLM, g.bn, a.dtype == MOE_DT_BF16, kMnA, kMnB);
      uint32_t ad = (uint32_t)ad0, phase = 0, count = 0;
      int slot = 0;
      bool ok = true, ready = false;        // ready: the next stage is known to have landed
      for (int u = first; ok && u < U; u += stride, ++count) {
        const int d = count & 1;
        if (!tc::mbar_wait(&accempty[d], ((count >> 1) & 1) ^ 1, abort)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t dt = tmem + d * 256;
        uint32_t acc = 0;
        for (int left = g.K; left > 0; left -= kLK) {
          if (!ready && !tc::bar_wait(full_u + 8 * slot, phase, abort)) { ok = false; break; }
          const uint32_t done = empty_u + 16 * slot, now = ad;
          ad += 2 * step;
          if (++slot == kLStages) {
            slot = 0;
            phase ^= 1;
            ad = (uint32_t)ad0;
          }
          // asked now, so that the answer's latency passes behind the MMAs' issue
          ready = tc::bar_test(full_u + 8 * slot, phase);
          tc::fence_after_sync();
          tc::mma_f16_x4<2>(dt, now, ahi, sa, now + b_off, bhi, sb, idesc, acc);
          tc::bar_commit_pair(done);
          acc = 1;
          if (left > kLH) tc::mma_f16_x4<2>(dt, now + step, ahi, sa, now + step + b_off, bhi, sb, idesc, 1u);
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
    uint16_t *z = reinterpret_cast<uint16_t*>(a.z), *out = g.out;
    const bool vo = rows16(out, g.ldo), vr = rows16(res, a.ldr), vz = rows16(z, a.ldz), vu = vz && a.N % 8 == 0;
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
      const int nr = (int)max((int64_t)0, min((int64_t)32, g.M - r0));
      const int cols = min(fn, g.N - tn * fn);
      constexpr bool kFwd = MODE == kLinFwd;
      float bl[kBlocks], bu[kBlocks];
#pragma unroll
      for (int i = 0; kFwd && i < kBlocks; ++i) {
        const int c = 32 * (wg + 2 * i) + lane;
        bl[i] = a.bias && c < cols ? bias((int64_t)tn * fn + c) : 0.f;
        bu[i] = GATED && a.bias && c < cols ? bias((int64_t)a.N + (int64_t)tn * fn + c) : 0.f;
      }
      uint4 ahead[4];       // the next block's residual, as block_in holds it
      const uint16_t* rp = res ? res + r0 * a.ldr + (int64_t)tn * fn : nullptr;
      auto fetch = [&](int c) {
        if (!kFwd || !res || !vr || c + 32 > cols) return;
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
          y[i] = __uint_as_float(v[i]);
          if constexpr (kFwd) y[i] += __shfl_sync(kFull, bl[blk], i);
          if constexpr (GATED) w[i] = __float_as_uint(__uint_as_float(w[i]) + __shfl_sync(kFull, bu[blk], i));
        }
        if (kFwd && z) {
          block_out<E>(st, z + r0 * a.ldz + n0, a.ldz, nr, nc, vz, lane, y);
          if constexpr (GATED) block_out<E>(st, z + r0 * a.ldz + a.N + n0, a.ldz, nr, nc, vu, lane, reinterpret_cast<float(&)[32]>(w));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if constexpr (GATED) y[i] = act_two(y[i], __uint_as_float(w[i]), a.act);
          else if constexpr (kFwd) y[i] = act_one(y[i], a.act.act);
        }
        if (kFwd && res) {
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
        block_out<E>(st, out + r0 * g.ldo + n0, g.ldo, nr, nc, vo, lane, y);
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

template <typename E, int MODE, bool GATED>
static cudaError_t launch_pairs(LinArgs& g, cudaStream_t st) {
  const LinearArgs& a = g.a;
  const auto kernel = k_linear<E, MODE, GATED>;
  // pairs that are resident at once, asked once per device
  static std::atomic<bool> done[kMaxDevices] = {};
  static std::atomic<int> pairs[kMaxDevices] = {};
  cudaError_t e = set_smem_once((const void*)kernel, kLSmem, done);
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
    if (cudaOccupancyMaxActiveClusters(&np, kernel, &cfg) != cudaSuccess || np <= 0) np = std::max(1, device_sms() / 2);
    if (slot) pairs[dev].store(np, std::memory_order_release);
  }
  // columns a tile: the width whose rounds over the pairs cost least. A half stage takes
  // its MMAs 2 bn cycles, and its copies, at 64 bytes a cycle, 2 for each row of x and
  // of the CTA's half of the columns, which is more but for the widest; a fixed part each
  constexpr int kStep = GATED ? 64 : 32;        // of the MMA: whole blocks of 32 columns of out
  g.mt = (int)up(g.M, 2 * kLM);
  int64_t least = INT64_MAX;
  for (int bn = 256; bn >= 64; bn -= kStep) {
    const int64_t nt = up(g.N, GATED ? bn / 2 : bn), copied = MODE == kLinFwd ? bn / 2 : up(bn / 2, 64) * 64;
    const int64_t cost = up(g.mt * nt, np) * (kLM + copied + 32);
    if (cost < least) {
      least = cost;
      g.bn = bn;
      g.nt = (int)nt;
    }
  }
  if ((int64_t)g.mt * g.nt >= (1ll << 31) - 4096) return cudaErrorInvalidValue;
  g.group = 8;
  LinMaps maps;
  bool ok;
  // K-major: boxes of 64 of the reduction x rows; else of 64 columns x 64 of the reduction
  auto rows = [&](CUtensorMap* map, const void* p, int64_t r, int64_t k, int64_t ld, int box) {
    const int64_t d[2] = {k, r}, sd[1] = {ld};
    const int b[2] = {kLH, box};
    return make_tmap(map, p, 2, 2, d, sd, b);
  };
  if constexpr (MODE == kLinFwd) {
    const int64_t wd[3] = {a.K, a.N, GATED ? 2 : 1}, ws[2] = {a.ldw, GATED ? (int64_t)a.N * a.ldw : a.ldw};
    const int wb[3] = {kLH, g.bn / 2, 1};
    ok = rows(&maps.x, a.x, a.R, a.K, a.ldx, kLM) && make_tmap(&maps.w, a.w, 2, 3, wd, ws, wb);
  } else if constexpr (MODE == kLinDx) {
    ok = rows(&maps.x, a.dz, a.R, g.K, a.lddz, kLM) && rows(&maps.w, a.w, g.K, a.K, a.ldw, kLH);
  } else {
    ok = rows(&maps.x, a.dz, a.R, g.M, a.lddz, kLH) && rows(&maps.w, a.x, a.R, a.K, a.ldx, kLH);
  }
  if (!ok) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(np, (int64_t)g.mt * g.nt));
  cfg.numAttrs = 2;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, g, maps);
}
// Whether a result of M x N (gated: of N columns a half) has tiles for about half of the pairs.
static bool for_pairs(int64_t M, int64_t N) { return up(M, 2 * kLM) * up(N, 64) >= 40; }

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t st) {
  const bool gated = act_gated(a.act.act);
  // Few rows, or too few columns for the pairs. 128 rows x 7168 x 2048 18 us here, 15 with
  // pairs, 96 rows x 2 x 2048 x 7168 21 and 31, 256 rows x 640 x 704 7 and 9.
  if (a.R <= 128 || (a.R <= kFewRows && !for_pairs(a.R, (int64_t)a.N * (gated ? 2 : 1)))) {
    FewArgs f = {};
    f.R = a.R; f.K1 = a.K; f.F1 = a.N; f.act = a.act; f.dtype = a.dtype; f.wdtype = a.wdtype; f.status = a.status;
    f.bias = a.bias; f.res = a.res; f.ldr = a.ldr; f.z = a.z; f.ldz = a.ldz; f.out = a.out; f.ldo = a.ldo;
    return launch_few_linear(f, a.x, a.ldx, a.w, a.ldw, st);
  }
  LinArgs g = {};
  g.a = a;
  g.M = a.R; g.N = a.N; g.K = a.K; g.out = reinterpret_cast<uint16_t*>(a.out); g.ldo = a.ldo;
  const bool bf = a.dtype == MOE_DT_BF16;
  if (gated) return bf ? launch_pairs<Bf16, kLinFwd, true>(g, st) : launch_pairs<F16, kLinFwd, true>(g, st);
  return bf ? launch_pairs<Bf16, kLinFwd, false>(g, st) : launch_pairs<F16, kLinFwd, false>(g, st);
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
  // The products: pairs of SMs where there are tiles for them, else the grouped
  // products' kernel with one group (narrow tiles, the reduction split).
  const bool bf = a.dtype == MOE_DT_BF16;
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
    if (a.R > 128 && for_pairs(a.R, a.K)) {
      g.M = a.R; g.N = a.K; g.K = rows; g.out = reinterpret_cast<uint16_t*>(a.dx); g.ldo = a.lddx;
      e = bf ? launch_pairs<Bf16, kLinDx, false>(g, st) : launch_pairs<F16, kLinDx, false>(g, st);
    } else {
      m.N = a.K; m.K = rows; m.b = a.w; m.ldb = a.ldw; m.trans_b = 1; m.out = a.dx; m.ldo = a.lddx;
      m.S = mm_splits(kMmRows, a.R, a.K, rows, 1);
      e = launch_mm16(m, false, st);
    }
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    if (a.R > 128 && for_pairs(rows, a.K)) {
      g.M = rows; g.N = a.K; g.K = a.R; g.out = reinterpret_cast<uint16_t*>(a.dw); g.ldo = a.lddw;
      return bf ? launch_pairs<Bf16, kLinDw, false>(g, st) : launch_pairs<F16, kLinDw, false>(g, st);
    }
    m.N = rows; m.K = a.K; m.b = a.x; m.ldb = a.ldx; m.trans_b = 0; m.out = a.dw; m.ldo = a.lddw; m.og = 0;
    m.S = mm_splits(kMmWgrad, a.R, rows, a.K, 1);
    return launch_mm16(m, true, st);
  }
  return cudaSuccess;
}

}  // namespace moe
