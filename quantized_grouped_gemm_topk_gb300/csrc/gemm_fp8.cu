// FP8 products with a scale for each block of 128, dense or grouped by expert:
//
//   out[r, n] = sum_b xs[r, b] ws[n / 128, b] sum_{k in block b} xq[r, k] wq[n, k]
//
// on the 5th-generation tensor cores (tcgen05.mma kind::f8f6f4, E4M3 operands
// in shared memory). The scales are arbitrary fp32 numbers, so the tensor
// core only sums inside a block: every 128 of K its accumulator starts anew,
// in one of 512 / BN tensor-memory slots, and the epilogue threads add it,
// times the block's scale, to the fp32 sums of the tile that they hold in
// registers. A thread's columns share one weight scale, so a block costs one
// multiply per row and one fused multiply-add per element, while the next
// blocks' MMAs run.
//
// Bound: the tensor pipe at training sizes (a 128 x 256 x 128 block is 512
// cycles of MMA, its additions 256 issue slots a scheduler at most), the
// weights' bytes at decode sizes.
// Measured: 8192^3 511 us (2.15 PFLOP/s; sustained, at the power limit, 546), 8192 x
// 7168 x 4096 237 us, 12289 rows in 32 equal groups x 4096 x 7168 358 us, in ragged
// ones 395, 3 x 7168 x 2048 10.7 us.
// At 8192^3 a block takes 1000 cycles; without the additions 816, without them
// and three of the four MMAs 670 (the copies: 48 KB at what an SM takes in).
// Of a block's way the issue of its MMAs is 600 cycles, the last commit's until
// the adding warps see it 680, the reads of tensor memory and the sums 460: the
// round trip of its slot is what shows, not the copies (a pair of SMs, with 32
// KB a block, took 512 us) nor power (all-zero operands 507).
// Tiles are 128 rows x BN columns on one SM; copies and edges as in gemm16.cu.
// Roles: warp 0 copies W, warp 2 copies x, warps 1 and 3 issue the MMAs of the
// tile's halves (warp 3 first clears rows outside every group), warps 4-11
// add: warp quarter q of tensor memory, half h of the columns (eight warps of
// 128 columns took 511 us there, sixteen of 64 columns 549). They take
// registers from the first four warps (setmaxnreg).
// Every wait is bounded, as in gemm16.cu.
#include "groups.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kFK = kQBlock;              // reduction a stage: one scale block, one 128-byte swizzle row
constexpr int kFThreads = 384;
constexpr int kFABytes = kGM * kFK;
constexpr int kFTables = 2 * 4 * (kMmMaxGroups + 1);
// Registers a thread: at launch, then of warps 0-3 and of warps 4-11. The
// shares sum to at most the launch's (checked against the built kernel
// before its first launch).
constexpr int kFRegs = 168, kFRegsLow = 80, kFRegsHigh = 208;
static_assert(128 * kFRegsLow + 256 * kFRegsHigh <= kFThreads * kFRegs, "register shares");

template <int BN>
struct FCfg {
  static constexpr int kBBytes = BN * kFK;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  // Tensor memory holds 512 / BN blocks' accumulators. A 256-wide tile runs as
  // two halves with an MMA issuer and slots of their own: the round trip of a
  // slot (MMA, commit, additions, release) is longer than the MMAs that two
  // slots queue, and half the columns halve its share of it.
  static constexpr int kHalves = BN == 256 ? 2 : 1;
  static constexpr int kHN = BN / kHalves;
  static constexpr int kSlots = 512 / BN;       // of each half
  static constexpr int kSmem = 1024 + kStages * (kFABytes + kBBytes) + 1024 + kFTables;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};
struct FMaps {
  CUtensorMap a[4];     // boxes of 16 << i rows
  CUtensorMap b;
};
struct FArgs {
  MmArgs m;
  int n_tiles;
};

struct GUnit {
  int e, row0, rows;    // first x row of the tile and its real rows
  int n0;               // first column
  int k0, k1;           // reduction blocks of a stage each: [k0, k1) of this piece
  int piece;
};

// Unit u: (row tile of a group, column tile, piece of the reduction), pieces
// innermost, then column tiles.
template <int BN>
__device__ __forceinline__ void f_unit(const MmArgs& m, int n_tiles, const int32_t* off, const int32_t* uoff, int u,
                                       GUnit& w) {
  const int S = m.S;
  const int t = u / S;
  w.piece = u - t * S;
  const int ui = t / n_tiles;
  w.n0 = (t - ui * n_tiles) * BN;
  w.e = group_of_unit(uoff, m.G, ui);
  const int mi = ui - uoff[w.e], cnt = off[w.e + 1] - off[w.e];
  w.row0 = off[w.e] + mi * kGM;
  w.rows = min(kGM, cnt - mi * kGM);
  const int nk = (m.K + kFK - 1) / kFK;
  w.k0 = (int)((int64_t)nk * w.piece / S);
  w.k1 = S == 1 ? nk : (int)((int64_t)nk * (w.piece + 1) / S);
}

// A copy of a tile's rows covers 16 << i of them, the fewest that hold its real
// ones; the MMA's other rows are an earlier stage's bytes and are not stored.
__device__ __forceinline__ int f_a_box(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

// Neither zero nor subnormal, infinite or NaN.
__device__ __forceinline__ bool normal(float v) {
  return (__float_as_uint(v) & 0x7fffffffu) - 0x00800000u < 0x7f000000u;
}

template <int BN>
__global__ void __launch_bounds__(kFThreads, 1) k_gemm_fp8(const FArgs g, const __grid_constant__ FMaps maps) {
  using C = FCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sa = base;
  uint8_t* sb = sa + C::kStages * kFABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + C::kStages * C::kBBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + C::kHalves * C::kSlots;      // of half h: [h * kSlots, ...)
  uint64_t* drain = tempty + C::kHalves * C::kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + C::kHalves);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tmp = reinterpret_cast<int*>(tmem_slot + 2);
  int32_t* off = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full) + 1024);
  int32_t* uoff = off + kMmMaxGroups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MmArgs& m = g.m;

  pdl_enter();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(&full[i], 2);
      tc::mbar_init(&empty[i], C::kHalves);
    }
    for (int i = 0; i < C::kHalves * C::kSlots; ++i) {
      tc::mbar_init(&tfull[i], 1);
      tc::mbar_init(&tempty[i], 8 / C::kHalves);     // one per adding warp
    }
    for (int i = 0; i < C::kHalves; ++i) tc::mbar_init(&drain[i], 1);
    *abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
  build_groups<kFThreads>(m.offsets, m.G, m.R, off, uoff, tmp, m.status, [](int c) { return (c + kGM - 1) / kGM; });
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int U = uoff[m.G] * g.n_tiles * m.S;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFRegsLow));
    // the single-thread loops below bound the whole where they are longer than
    // the MMAs: addresses and parities are carried along, not computed
    const uint32_t full_u = tc::smem_u32(full), empty_u = tc::smem_u32(empty);
    const uint32_t sa_u = tc::smem_u32(sa), sb_u = tc::smem_u32(sb);
    if (warp == 0 || warp == 2) {
      // ---------------- copies: warp 0 W, warp 2 x ----------------
      if (lane == 0) {
        const bool isb = warp == 0;
        const uint32_t dst0 = isb ? sb_u : sa_u, step = isb ? C::kBBytes : kFABytes;
        int slot = 0;
        uint32_t phase = 1, issued = 0;          // of empty: the ring starts free
        bool ok = true;
        for (int u = blockIdx.x; ok && u < U; u += gridDim.x) {
          GUnit w;
          f_unit<BN>(m, g.n_tiles, off, uoff, u, w);
          const int ai = f_a_box(w.rows);
          const uint32_t bytes = isb ? C::kBBytes : (uint32_t)(kFK * (16 << ai));
          for (int kb = w.k0; kb < w.k1; ++kb) {
            if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
            const uint32_t bar = full_u + 8 * slot;
            tc::bar_arrive_expect_tx(bar, bytes);
            if (isb) tc::tma_load_3d_at(dst0 + slot * step, &maps.b, kb * kFK, w.n0, w.e, bar);
            else tc::tma_load_2d_at(dst0 + slot * step, &maps.a[ai], kb * kFK, w.row0, bar);
            ++issued;
            if (++slot == C::kStages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok || *abort) {        // wind-down: bounded waits for the copies in flight
          volatile int never = 0;
          const uint32_t n = issued < (uint32_t)C::kStages ? issued : (uint32_t)C::kStages;
          for (uint32_t k = 0; k < n; ++k) {
            const uint32_t i2 = issued - 1 - k;
            tc::mbar_wait(&full[i2 % C::kStages], (i2 / C::kStages) & 1, &never, 100000000ll);
          }
        }
      }
    } else {
      if (warp == 3) clear_rows_outside(m, off, lane);
      // ---------------- MMAs: warp 1 the first half, warp 3 the second ----------------
      const int h = warp >> 1;
      if (lane == 0 && h < C::kHalves) {
        // kind::f8f6f4: E4M3 is format 0 of both operands; fp32 accumulator
        constexpr uint32_t idesc = tc::idesc_f16_f32(kGM, C::kHN);
        const uint32_t tfull_u = tc::smem_u32(tfull + h * C::kSlots), tempty_u = tc::smem_u32(tempty + h * C::kSlots);
        const uint64_t ad0 = tc::smem_desc_sw128(sa_u), bd0 = tc::smem_desc_sw128(sb_u + h * C::kHN * kFK);
        uint64_t ad = ad0, bd = bd0;
        uint32_t slot_b = 0, phase = 0;          // the stage's barriers' offset, its parity
        uint32_t ts_b = 0, tphase = 1;           // the same of the accumulator's
        const uint32_t t0 = tmem + h * C::kHN;
        uint32_t dt = t0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < U; u += gridDim.x) {
          GUnit w;
          f_unit<BN>(m, g.n_tiles, off, uoff, u, w);
          for (int n = w.k1 - w.k0; n > 0; --n) {
            if (!tc::bar_wait(full_u + slot_b, phase, abort)) { ok = false; break; }
            if (!tc::bar_wait(tempty_u + ts_b, tphase, abort)) { ok = false; break; }
            tc::fence_after_sync();
#pragma unroll
            for (int j = 0; j < 4; ++j)     // K = 32: 32 bytes along the rows; past K both read as zero
              tc::mma_f8_ss(dt, ad + 2 * j, bd + 2 * j, idesc, j > 0 ? 1u : 0u);
            tc::bar_commit(tfull_u + ts_b);
            tc::bar_commit(empty_u + slot_b);
            ad += kFABytes / 16;
            bd += C::kBBytes / 16;
            slot_b += 8;
            if (slot_b == 8 * C::kStages) {
              slot_b = 0;
              phase ^= 1;
              ad = ad0;
              bd = bd0;
            }
            ts_b += 8;
            dt += BN;
            if (ts_b == 8 * C::kSlots) {
              ts_b = 0;
              tphase ^= 1;
              dt = t0;
            }
          }
        }
        tc::mma_commit(&drain[h]);
        volatile int never = 0;
        tc::mbar_wait(&drain[h], 0, &never, 400000000ll);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFRegsHigh));
    // ---------------- sums of the blocks ----------------
    constexpr int kCols = BN / 2, kChunks = kCols / 16;
    const int h = (warp - 4) >> 2, q = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + h * kCols;
    const uint32_t hfull = tc::smem_u32(tfull + h * C::kHalves / 2 * C::kSlots);
    const uint32_t hempty = tc::smem_u32(tempty + h * C::kHalves / 2 * C::kSlots);
    uint32_t ts = 0, tphase = 0;       // the accumulator's slot and parity
    const int KB = (m.K + kFK - 1) / kFK, NB = (m.N + kQBlock - 1) / kQBlock;
    const int dt = m.S > 1 ? MOE_DT_F32 : m.out_dtype;
    const int esize = dt == MOE_DT_F32 ? 4 : 2;
    const int64_t ld = m.S > 1 ? m.N : m.ldo, os = (int64_t)m.R * m.N;
    uint8_t* obase = reinterpret_cast<uint8_t*>(m.S > 1 ? (void*)m.part : m.out);
    const bool vec = ((uintptr_t)obase & 15) == 0 && (ld * esize) % 16 == 0 && (m.S == 1 || (os * 4) % 16 == 0);
    const int r = q * 32 + lane;
    bool ok = true;
    GUnit w;
    const float *xs = nullptr, *ws = nullptr;
    // The scales of the next four blocks are on their way, each in registers
    // of its own: a copy from register to register would wait for the load. A
    // tile's first ones are loaded before the last tile is stored.
    float s[4], t[4];
    auto begin = [&](int u) {
      f_unit<BN>(m, g.n_tiles, off, uoff, u, w);
      xs = m.sa + (int64_t)(w.row0 + (r < w.rows ? r : 0)) * m.ldsa;
      const int nb = min((w.n0 + h * kCols) / kQBlock, NB - 1);     // past N: nothing is stored
      ws = m.sb + ((int64_t)w.e * NB + nb) * KB;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = w.k0 + j < w.k1;
        s[j] = in ? xs[w.k0 + j] : 0.f;
        t[j] = in ? ws[w.k0 + j] : 0.f;
      }
    };
    if ((int)blockIdx.x < U) begin(blockIdx.x);
    for (int u = blockIdx.x; u < U; u += gridDim.x) {
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      // acc += f1 x (TWICE: f0 x) the block's sums, and the slot is released
      auto add_block = [&](auto twice, float f0, float f1) {
        const uint32_t at = lanes + ts * BN;
        // chunk c + 1 is read while chunk c is added
        uint32_t v[2][16];
        tc::tmem_ld16(at, v[0]);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          tc::tmem_wait_ld();
          if (c + 1 < kChunks) {
            tc::tmem_ld16(at + 16 * (c + 1), v[(c + 1) & 1]);
          } else {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(hempty + 8 * ts);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(v[c & 1][i]);
            acc[c * 16 + i] = fmaf(decltype(twice)::value ? x * f0 : x, f1, acc[c * 16 + i]);
          }
        }
      };
      // Scales whose product leaves fp32's normal range though its product with
      // the sum need not (0 x inf would be NaN, a subnormal would cut digits):
      // one after the other, the intermediate in range, by the smaller first
      // where the product is large and by the larger where it is small. Other
      // rows of the warp keep their bits.
      auto add_odd_block = [&](float a, float b) {
        const float sc = a * b;
        const bool a_first = (fabsf(a) > fabsf(b)) != (fabsf(sc) > 1.f), one = normal(sc);
        add_block(std::true_type(), one ? 1.f : a_first ? a : b, one ? sc : a_first ? b : a);
      };
      for (int kb0 = w.k0; kb0 < w.k1; kb0 += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int kb = kb0 + j;
          if (kb < w.k1 && ok) {
            const float sc = s[j] * t[j];
            const bool odd = __any_sync(kFull, !normal(sc));
            if (kb + 4 < w.k1) {
              s[j] = xs[kb + 4];
              t[j] = ws[kb + 4];
            }
            ok = __all_sync(kFull, tc::bar_wait_inline(hfull + 8 * ts, tphase, abort));
            if (ok) {
              tc::fence_after_sync();
              if (!odd) add_block(std::false_type(), 1.f, sc);
              else add_odd_block(xs[kb], ws[kb]);
              if (++ts == C::kSlots) {
                ts = 0;
                tphase ^= 1;
              }
            }
          }
        }
      }
      if (!ok) break;
      const int col = w.n0 + h * kCols, rows = w.rows - q * 32;
      const int64_t row = (int64_t)(w.row0 + q * 32) * ld + (m.S > 1 ? w.piece * os : 0);
      if (u + (int)gridDim.x < U) begin(u + gridDim.x);
      if (vec && col + kCols <= m.N) {
        store_block<kCols>(obase + (row + col) * esize, ld * esize, acc, rows, lane, dt);
      } else if (lane < rows) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (col + 16 * c < m.N) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(acc[c * 16 + i]);
            store_cols(obase + (row + lane * ld + col + 16 * c) * esize, v, m.N - col - 16 * c, dt, vec);
          }
        }
      }
      __syncwarp();
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) set_status(m.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---- host -------------------------------------------------------------------------
template <int BN>
static cudaError_t launch_f(FArgs g, cudaStream_t st) {
  using C = FCfg<BN>;
  const MmArgs& m = g.m;
  FMaps maps;
  for (int i = 0; i < 4; ++i) {
    const int64_t dims[2] = {m.K, m.R}, strides[1] = {m.lda};
    const int box[2] = {kFK, 16 << i};
    if (!make_tmap(&maps.a[i], m.a, 1, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const int64_t dims[3] = {m.K, m.N, m.G}, strides[2] = {m.ldb, m.G > 1 ? m.bg : m.ldb};
  const int box[3] = {kFK, BN, 1};
  if (!make_tmap(&maps.b, m.b, 1, 3, dims, strides, box)) return cudaErrorInvalidValue;
  g.n_tiles = (m.N + BN - 1) / BN;
  // a kernel launched with fewer registers than its warps then share out
  // would wait for them forever
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, k_gemm_fp8<BN>);
    if (e != cudaSuccess) return e;
    regs.store(at.numRegs, std::memory_order_release);
  }
  if (128 * kFRegsLow + 256 * kFRegsHigh > kFThreads * regs.load()) return cudaErrorInvalidConfiguration;
  if (!units_fit(m, m.R / kGM, g.n_tiles)) return cudaErrorInvalidValue;
  static std::atomic<bool> done[kMaxDevices] = {};
  cudaError_t e = set_smem_once((const void*)k_gemm_fp8<BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_pdl(k_gemm_fp8<BN>, dim3(device_sms()), dim3(kFThreads), C::kSmem, st, g, maps);
  if (e != cudaSuccess || m.S == 1) return e;
  return launch_mm_join(m, false, st);
}

cudaError_t launch_mm_fp8(const MmArgs& a, cudaStream_t st) {
  FArgs g = {};
  g.m = a;
  const int bn = mm_plan(kMmFp8, a.R, a.N, a.K, a.G).bn;
  return bn == 256 ? launch_f<256>(g, st) : bn == 128 ? launch_f<128>(g, st) : launch_f<64>(g, st);
}

}  // namespace moe
