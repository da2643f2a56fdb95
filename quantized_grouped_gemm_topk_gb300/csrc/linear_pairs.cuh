// The dense products of many rows: tcgen05 on pairs of SMs (cta_group::2), tiles of 256 rows of
// x (the MMA's M, a lane of tensor memory each) by up to 256 columns. Rows on the
// M side, unlike the grouped products: a thread then holds neighbouring columns of
// one row, and of a gated tile (as many gate as up columns: the first CTA of the
// pair copies the gate's weights, the second the up's) both halves of each of its
// outputs, so the activation needs no exchange. Few rows: few16.cu. The backward's
// products run in the same kernel, dw with dz's columns as M, and with the operands
// whose M or N axis is contiguous in memory (w for dx, both for dw) as they lie there.
//
// Bound: many rows, the tensor cores, and under load the power limit; few tiles, the
// way along the reduction (one tile a pair), launch and the epilogue behind it.
// Measured, bf16, in us: 16384 x 2 x 2880 x 2880 with z 301 (1.81 PFLOP/s), 16384 x 7168 x 4096 with residual
// 511 (1.88), dx and dw of 16384 x 2 x 2880 x 2880 315 and 325 (1.73, 1.67); 4096 rows: tensor pipe 73 to 77 %
// busy. 333 x 2880 x 1984 f16 with bias, GELU, residual and z 14.9, with rows that start off 16
// bytes (VEC = false) 17.3; without any of the four 12.4.
#pragma once
#include "linear.cuh"
#include "tc.cuh"

namespace moe {

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

struct LinMaps {
  CUtensorMap x, w;     // the operands A and B
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
// memory; VEC: rows start on 16 bytes.
// Such a block on its way in: asked for, and put into staging memory. VEC: four
// 16-byte units a lane; else (any alignment, or fewer columns) a column a lane.
template <bool VEC>
struct BlockIn {
  uint4 u[VEC ? 4 : 1];
  uint16_t v[VEC ? 1 : 32];
  __device__ __forceinline__ void fetch(const uint16_t* p, int64_t ld, int nr, int nc, int lane) {
    if constexpr (VEC) {
      if (nc < 32) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (lane >> 2) + 8 * i;
        if (row < nr) u[i] = *reinterpret_cast<const uint4*>(p + row * ld + 8 * (lane & 3));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = i < nr && lane < nc ? p[i * ld + lane] : (uint16_t)0;
    }
  }
  __device__ __forceinline__ void put(uint8_t* st, const uint16_t* p, int64_t ld, int nr, int nc, int lane) const {
    if constexpr (VEC) {
      if (nc < 32) {
#pragma unroll 8
        for (int i = 0; i < 32; ++i)
          if (i < nr && lane < nc) *reinterpret_cast<uint16_t*>(st + i * kLRow + 2 * lane) = p[i * ld + lane];
        return;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(st + ((lane >> 2) + 8 * i) * kLRow + 16 * (lane & 3)) = u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) *reinterpret_cast<uint16_t*>(st + i * kLRow + 2 * lane) = v[i];
    }
  }
};
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
template <typename E, bool VEC>
__device__ __forceinline__ void block_out(uint8_t* st, uint16_t* p, int64_t ld, int nr, int nc, int lane, const float (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(st + lane * kLRow + 16 * i) =
        make_uint4(E::from2(r[8 * i], r[8 * i + 1]), E::from2(r[8 * i + 2], r[8 * i + 3]), E::from2(r[8 * i + 4], r[8 * i + 5]),
                   E::from2(r[8 * i + 6], r[8 * i + 7]));
  __syncwarp();
  if (VEC && nc >= 32) {
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

// The activation, known to the compiler, of 32 columns, or of 16 pairs.
template <int ACT>
__device__ __forceinline__ void act_all(float (&y)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) y[i] = act_one(y[i], ACT);
}
template <int ACT>
__device__ __forceinline__ void act_all(float* y, const uint32_t (&g)[16], const uint32_t (&u)[16], const ActParams& p) {
  const ActParams act = {ACT, p.alpha, p.limit};
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = act_two(__uint_as_float(g[i]), __uint_as_float(u[i]), act);
}

template <typename E, int MODE, bool GATED, bool VEC>
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
    auto bias = [&](int64_t f) {
      return a.wdtype == MOE_DT_F32 ? reinterpret_cast<const float*>(a.bias)[f] : E::to(reinterpret_cast<const uint16_t*>(a.bias)[f]);
    };
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
      float bl = 0.f, bu = 0.f;         // the next block's biases, a column a lane
      auto fetch_bias = [&](int c) {
        if (!kFwd || !a.bias || c + lane >= cols) return;
        bl = bias((int64_t)tn * fn + c + lane);
        if (GATED) bu = bias((int64_t)a.N + (int64_t)tn * fn + c + lane);
      };
      // the next block's residual; not ahead of a gated block, whose halves take the registers
      BlockIn<VEC> ahead;
      const uint16_t* rp = res ? res + r0 * a.ldr + (int64_t)tn * fn : nullptr;
      auto fetch = [&](int c) {
        if (kFwd && res && c < cols) ahead.fetch(rp + c, a.ldr, nr, min(32, cols - c), lane);
      };
      fetch_bias(32 * wg);
      if (!GATED) fetch(32 * wg);
      const bool got = tc::mbar_wait(&accfull[d], (count >> 1) & 1, abort);
      if (!__all_sync(kFull, got)) break;
      tc::fence_after_sync();
#pragma unroll 1
      for (int c = 32 * wg; c < cols; c += 64) {
        const int nc = min(32, cols - c);
        const int64_t n0 = (int64_t)tn * fn + c;
        float y[32];
        // 32 columns of the accumulator with their biases
        auto load = [&](uint32_t col, float bias) {
          uint32_t v[32];
          tc::tmem_ld32(acc + col, v);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(v[i]) + (kFwd ? __shfl_sync(kFull, bias, i) : 0.f);
        };
        if constexpr (!GATED) {
          load(c, bl);
          if (kFwd && z) block_out<E, VEC>(st, z + r0 * a.ldz + n0, a.ldz, nr, nc, lane, y);
          if constexpr (kFwd) {
            if (a.act.act == MOE_ACT_GELU) act_all<MOE_ACT_GELU>(y);
            else if (a.act.act == MOE_ACT_SILU) act_all<MOE_ACT_SILU>(y);
            else if (a.act.act == MOE_ACT_SRELU) act_all<MOE_ACT_SRELU>(y);
          }
        } else {
          // read again for the activation, in two halves: registers are the scarcer
          if (z) {
            load(c, bl);
            block_out<E, VEC>(st, z + r0 * a.ldz + n0, a.ldz, nr, nc, lane, y);
            load(fn + c, bu);
            block_out<E, VEC>(st, z + r0 * a.ldz + a.N + n0, a.ldz, nr, nc, lane, y);
          }
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            uint32_t v[16], w[16];
            tc::tmem_ld16(acc + c + h, v);
            tc::tmem_ld16(acc + fn + c + h, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = __float_as_uint(__uint_as_float(v[i]) + __shfl_sync(kFull, bl, h + i));
              w[i] = __float_as_uint(__uint_as_float(w[i]) + __shfl_sync(kFull, bu, h + i));
            }
            if (a.act.act == MOE_ACT_SWIGLU) act_all<MOE_ACT_SWIGLU>(y + h, v, w, a.act);
            else if (a.act.act == MOE_ACT_GEGLU) act_all<MOE_ACT_GEGLU>(y + h, v, w, a.act);
            else act_all<MOE_ACT_SWIGLU_CLAMP>(y + h, v, w, a.act);
          }
        }
        fetch_bias(c + 64);
        if (kFwd && res) {
          if (GATED) fetch(c);
          ahead.put(st, rp + c, a.ldr, nr, nc, lane);
          if (!GATED) fetch(c + 64);
          add_row<E>(st, lane, y);
        }
        block_out<E, VEC>(st, out + r0 * g.ldo + n0, g.ldo, nr, nc, lane, y);
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


template <typename E, int MODE, bool GATED, bool VEC>
static cudaError_t launch_pairs(LinArgs& g, cudaStream_t st) {
  const LinearArgs& a = g.a;
  const auto kernel = k_linear<E, MODE, GATED, VEC>;
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
  // Column tiles innermost where all their operand stays in L2; else eight row tiles
  // share each column tile (16384 x 2 x 2880 x 2880, 33 MB of weights, 298 us and 305;
  // 16384 x 7168 x 4096, 59 MB, 546 and 513).
  g.group = (int64_t)g.nt * g.bn * g.K * 2 <= (40ll << 20) ? 1 : 8;
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

template <typename E>
static cudaError_t launch_pairs(LinArgs& g, int mode, bool gated, cudaStream_t st) {
  const LinearArgs& a = g.a;
  const bool fwd = mode == kLinFwd;
  const bool vec = rows16(g.out, g.ldo) && (!fwd || ((!a.res || rows16(a.res, a.ldr)) && (!a.z || (rows16(a.z, a.ldz) && (!gated || a.N % 8 == 0)))));
  if (mode == kLinDx) return vec ? launch_pairs<E, kLinDx, false, true>(g, st) : launch_pairs<E, kLinDx, false, false>(g, st);
  if (mode == kLinDw) return vec ? launch_pairs<E, kLinDw, false, true>(g, st) : launch_pairs<E, kLinDw, false, false>(g, st);
  if (gated) return vec ? launch_pairs<E, kLinFwd, true, true>(g, st) : launch_pairs<E, kLinFwd, true, false>(g, st);
  return vec ? launch_pairs<E, kLinFwd, false, true>(g, st) : launch_pairs<E, kLinFwd, false, false>(g, st);
}

}  // namespace moe
