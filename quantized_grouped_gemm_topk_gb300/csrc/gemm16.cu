// Products grouped by expert with ragged sizes, bf16 or f16, on the
// 5th-generation tensor cores (tcgen05.mma kind::f16, operands in shared
// memory, fp32 accumulators in tensor memory).
//
//   kRowsNT   out[r] = W_e x[r]      A = x rows, B = W rows; both K-major
//   kRowsNN   out[r] = W_e^T x[r]    B has its N axis contiguous (the
//             gradient of the rows with the forward's weights, no transpose)
//   kWgrad    dW_e = sum over group rows dy[r]^T x[r]; both operands have
//             their M / N axis contiguous and the reduction runs over rows
//
// Bound: the tensor pipe at training sizes (2 R N K FLOPs), the weights'
// bytes at decode sizes. Tiles: 128 rows x BN columns (256; 128 or 64 where
// larger tiles would leave SMs without work) x 64 of the reduction a stage,
// in a ring that fills the shared memory, filled by tensor copies with the
// 128-byte swizzle and drained by four MMAs of K = 16. Ragged edges cost no
// branch in the main loop: rows of a tile that belong to the next group only
// reach accumulator rows that are not stored; columns and the K tail read as
// zeros (the tensor maps end at N and K); the weight gradient's last rows are
// cleared in shared memory, both operands (a NaN of the next group times zero
// would be NaN).
//
// Roles (one CTA per SM, persistent over the units): warp 0 copies B, warp 2
// copies A (two issuers: a copy costs its thread some hundred cycles), warp 1
// issues the MMAs, warps 4-7 and 8-11 are epilogues that alternate between
// tiles and the two accumulators, so a tile's stores overlap the next one's
// MMAs; warp 3 clears rows outside every group.
// Every wait is bounded; a CTA whose wait runs out sets MOE_DEV_TIMEOUT, waits
// for its copies and MMAs in flight, frees tensor memory and returns.
#include "groups.cuh"
#include "tc.cuh"

namespace moe {

enum { kRowsNT = 0, kRowsNN = 1, kWgradMN = 2 };

constexpr int kGK = 64;               // reduction a stage: one 128-byte swizzle row
constexpr int kGThreads = 384;
constexpr int kGChunk = 64 * kGK * 2; // bytes of 64 M / N elements of an MN-contiguous stage
constexpr int kGABytes = kGM * kGK * 2;
constexpr int kGTables = 2 * 4 * (kMmMaxGroups + 1);

template <int BN>
struct GCfg {
  static constexpr int kBBytes = BN * kGK * 2;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr int kSmem = 1024 + kStages * (kGABytes + kBBytes) + 1024 + kGTables;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

struct GMaps {
  CUtensorMap a[4];     // K-major A: boxes of 16 << i rows; MN: a[0]
  CUtensorMap b;
};
struct GArgs {
  MmArgs m;
  int n_tiles;          // BN-wide column tiles
  int m_tiles;          // wgrad: 128-row tiles of N
  int a_chunks, b_chunks;   // MN-contiguous operands: 64-wide chunks a copy takes (1: one copy a chunk)
};

// Copies of one MN-contiguous operand stage: `chunks` chunks of 64 columns
// from column c0, rows row0 .. row0 + 63 of matrix z.
__device__ __forceinline__ void g_load_mn(uint8_t* dst, const CUtensorMap* map, int c0, int row0, int z, int chunks,
                                          int per_copy, uint64_t* bar) {
  if (per_copy > 1) {
    tc::tma_load_4d_plain(dst, map, 0, row0, c0 / 64, z, bar);
  } else {
    for (int c = 0; c < chunks; ++c) tc::tma_load_4d_plain(dst + c * kGChunk, map, c0 + 64 * c, row0, 0, z, bar);
  }
}

template <int MODE, int BN>
__global__ void __launch_bounds__(kGThreads, 1) k_gemm16(const GArgs g, const __grid_constant__ GMaps maps) {
  using C = GCfg<BN>;
  constexpr bool kWg = MODE == kWgradMN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sa = base;
  uint8_t* sb = sa + C::kStages * kGABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + C::kStages * C::kBBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* accfull = empty + C::kStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tmp = reinterpret_cast<int*>(tmem_slot + 2);
  int32_t* off = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full) + 1024);
  int32_t* uoff = off + kMmMaxGroups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MmArgs& m = g.m;

  pdl_enter();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(&full[i], 2);       // one arrival (with its bytes) from each copying warp
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], 1);
      tc::mbar_init(&accempty[i], 4);   // one per epilogue warp
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, C::kTmemCols);
  build_groups<kGThreads>(m.offsets, m.G, m.R, off, uoff, tmp, m.status,
                          [&](int c) { return kWg ? g.m_tiles : (c + kGM - 1) / kGM; });
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int U = uoff[m.G] * g.n_tiles * m.S;

  if (warp == 0 || warp == 2) {
    // ---------------- copies: warp 0 B, warp 2 A ----------------
    if (lane == 0) {
      const bool isb = warp == 0;
      if (isb) tc::prefetch_tmap(&maps.b);
      else
        for (int i = 0; i < (kWg ? 1 : 4); ++i) tc::prefetch_tmap(&maps.a[i]);
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < U; u += gridDim.x) {
        GUnit w;
        g_unit<kWg, BN, kGK>(m, g.n_tiles, off, uoff, u, w);
        const int ai = g_a_box(w.rows);
        for (int kb = w.k0; kb < w.k1; ++kb, ++it) {
          const int slot = it % C::kStages;
          if (!tc::mbar_wait(&empty[slot], ((it / C::kStages) & 1) ^ 1, abort)) { ok = false; break; }
          if (isb) {
            uint8_t* d = sb + slot * C::kBBytes;
            tc::mbar_arrive_expect_tx(&full[slot], C::kBBytes);
            if (MODE == kRowsNT) tc::tma_load_3d_plain(d, &maps.b, kb * kGK, w.n0, w.e, &full[slot]);
            else if (MODE == kRowsNN) g_load_mn(d, &maps.b, w.n0, kb * kGK, w.e, BN / 64, g.b_chunks, &full[slot]);
            else g_load_mn(d, &maps.b, w.n0, off[w.e] + kb * kGK, 0, BN / 64, g.b_chunks, &full[slot]);
          } else {
            uint8_t* d = sa + slot * kGABytes;
            if (kWg) {
              tc::mbar_arrive_expect_tx(&full[slot], kGABytes);
              g_load_mn(d, &maps.a[0], w.row0, off[w.e] + kb * kGK, 0, kGM / 64, g.a_chunks, &full[slot]);
            } else {
              tc::mbar_arrive_expect_tx(&full[slot], (uint32_t)(kGK * 2 * (16 << ai)));
              tc::tma_load_2d_plain(d, &maps.a[ai], kb * kGK, w.row0, &full[slot]);
            }
          }
        }
      }
      if (!ok || *abort) {
        // wind-down: wait (bounded, ignoring the abort flag) for the copies
        // this thread still has in flight. A slot's barrier completes only
        // when the other copying warp arrived too; it may have stopped
        // earlier, so the wait's limit is what ends this then.
        volatile int never = 0;
        const uint32_t n = it < (uint32_t)C::kStages ? it : (uint32_t)C::kStages;
        for (uint32_t k = 0; k < n; ++k) {
          const uint32_t i2 = it - 1 - k;
          tc::mbar_wait(&full[i2 % C::kStages], (i2 / C::kStages) & 1, &never, 100000000ll);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    const uint32_t idesc = tc::idesc_16bit(kGM, BN, m.dtype == MOE_DT_BF16, kWg, MODE != kRowsNT);
    uint32_t it = 0, tcount = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < U; u += gridDim.x, ++tcount) {
      GUnit w;
      g_unit<kWg, BN, kGK>(m, g.n_tiles, off, uoff, u, w);
      const int d = tcount & 1;
      ok = __all_sync(kFull, tc::mbar_wait(&accempty[d], ((tcount >> 1) & 1) ^ 1, abort));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t dt = tmem + d * BN;
      for (int kb = w.k0; kb < w.k1; ++kb, ++it) {
        const int slot = it % C::kStages;
        ok = __all_sync(kFull, tc::mbar_wait(&full[slot], (it / C::kStages) & 1, abort));
        if (!ok) break;
        uint8_t* pa = sa + slot * kGABytes;
        uint8_t* pb = sb + slot * C::kBBytes;
        const int left = w.red - kb * kGK;          // of the reduction in this stage
        const int steps = left >= kGK ? 4 : (left + 15) / 16;
        if (kWg && left < kGK && (left & 15)) {
          // rows of the next group behind the last ones: cleared up to the
          // MMA's K, a 128-byte line per row and chunk (the swizzle permutes
          // within a line)
          const int bad = 16 - (left & 15);
          for (int i = lane; i < bad * 8 * (kGM / 64 + BN / 64); i += 32) {
            const int q = i & 7, r = left + (i >> 3) % bad, c = (i >> 3) / bad;
            uint8_t* line = (c < kGM / 64 ? pa + c * kGChunk : pb + (c - kGM / 64) * kGChunk) + r * 128;
            reinterpret_cast<uint4*>(line)[q] = make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        if (lane == 0) {
          tc::fence_after_sync();
          const uint64_t ad = kWg ? tc::smem_desc_mn_sw128(tc::smem_u32(pa), kGChunk) : tc::smem_desc_sw128(tc::smem_u32(pa));
          const uint64_t bd = MODE != kRowsNT ? tc::smem_desc_mn_sw128(tc::smem_u32(pb), kGChunk)
                                              : tc::smem_desc_sw128(tc::smem_u32(pb));
          // a step of K = 16: 32 bytes along a K-major row, two 8-row atoms otherwise
          constexpr uint32_t sta = kWg ? 2048 / 16 : 32 / 16, stb = MODE != kRowsNT ? 2048 / 16 : 32 / 16;
          for (int j = 0; j < steps; ++j)
            tc::mma_f16_ss(dt, ad + sta * j, bd + stb * j, idesc, (kb > w.k0 || j > 0) ? 1u : 0u);
          tc::mma_commit(&empty[slot]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) tc::mma_commit(&accfull[d]);
      __syncwarp();
    }
    if (lane == 0) {
      tc::mma_commit(drain);              // every MMA of this thread has completed once it fires
      volatile int never = 0;
      tc::mbar_wait(drain, 0, &never, 400000000ll);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------- rows outside every group ----------------
    if (!kWg) clear_rows_outside(m, off, lane);
  } else {
    // ---------------- epilogue ----------------
    const int wg = (warp - 4) >> 2, q = warp & 3;
    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + wg * BN;
    const int cols = kWg ? m.K : m.N;
    const int dt = m.S > 1 ? MOE_DT_F32 : m.out_dtype;
    const int esize = dt == MOE_DT_F32 ? 4 : 2;
    const int64_t ld = m.S > 1 ? cols : m.ldo;
    uint8_t* obase = reinterpret_cast<uint8_t*>(m.S > 1 ? (void*)m.part : m.out);
    const int64_t og = m.S > 1 ? (int64_t)m.N * m.K : m.og;
    const int64_t os = kWg ? (int64_t)m.G * m.N * m.K : (int64_t)m.R * m.N;      // a piece's partial sums
    const bool vec = ((uintptr_t)obase & 15) == 0 && (ld * esize) % 16 == 0 && (og * esize) % 16 == 0 &&
                     (m.S == 1 || (os * 4) % 16 == 0);
    uint32_t tcount = 0, mine = 0;
    for (int u = blockIdx.x; u < U; u += gridDim.x, ++tcount) {
      if ((int)(tcount & 1) != wg) continue;
      GUnit w;
      g_unit<kWg, BN, kGK>(m, g.n_tiles, off, uoff, u, w);
      const bool got = tc::mbar_wait(&accfull[wg], mine & 1, abort);
      if (!__all_sync(kFull, got)) break;
      tc::fence_after_sync();
      const int r = q * 32 + lane;
      int64_t at = kWg ? w.e * og + (int64_t)(w.row0 + r) * ld : (int64_t)(w.row0 + r) * ld;
      if (m.S > 1) at += w.piece * os;
      for (int c0 = 0; c0 < BN && w.n0 + c0 < cols; c0 += 32) {
        uint32_t v[32];
        if (w.k1 > w.k0) {
          tc::tmem_ld32(acc + c0, v);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;       // no rows to sum over
        }
        if (r < w.rows) store_cols(obase + (at + w.n0 + c0) * esize, v, cols - w.n0 - c0, dt, vec);
        __syncwarp();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&accempty[wg]);
      ++mine;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) set_status(m.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// out row i = the S partial sums of its elements, added in order; the rows of
// `rows` x `cols` partial matrices lie back to back, those of out at ldo
// (og between groups of rpg rows).
__global__ void __launch_bounds__(256) k_mm_join(const float* __restrict__ part, int S, int64_t rows, int cols,
                                                 int64_t rpg, void* out, int64_t ldo, int64_t og, int dtype) {
  pdl_enter();
  const int64_t n = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float v = part[i];
    for (int s = 1; s < S; ++s) v += part[s * n + i];
    const int64_t r = i / cols, gr = r / rpg;
    const int64_t at = gr * og + (r - gr * rpg) * ldo + (i - r * cols);
    if (dtype == MOE_DT_F32) reinterpret_cast<float*>(out)[at] = v;
    else reinterpret_cast<uint16_t*>(out)[at] = dtype == MOE_DT_F16 ? F16::from(v) : Bf16::from(v);
  }
}

cudaError_t launch_mm_join(const MmArgs& a, bool wgrad, cudaStream_t st) {
  const int64_t rows = wgrad ? (int64_t)a.G * a.N : a.R;
  const int cols = wgrad ? a.K : a.N;
  const int64_t blocks = std::min<int64_t>((rows * cols + 255) / 256, (int64_t)device_sms() * 8);
  note_launch();
  return launch_pdl(k_mm_join, dim3((unsigned)blocks), dim3(256), 0, st, (const float*)a.part, a.S, rows, cols,
                    wgrad ? (int64_t)a.N : rows, a.out, a.ldo, a.og, a.out_dtype);
}

// ---- sizes to tiles -------------------------------------------------------------
// The split rule must not depend on the device a size query runs on.
constexpr int kPlanSms = 152;
constexpr int64_t kPartBytes = 64ll << 20;

MmPlan mm_plan(int kind, int R, int N, int K, int G) {
  const bool wg = kind == kMmWgrad;
  // row tiles: at least one for every group that can have rows
  const int64_t mt = wg ? (int64_t)G * ((N + kGM - 1) / kGM)
                        : std::max<int64_t>((R + kGM - 1) / kGM, std::min(G, R));
  const int cols = wg ? K : N;
  const int64_t red = wg ? (R + G - 1) / G : K;
  MmPlan p;
  p.bn = 256;
  auto units = [&] { return mt * ((cols + p.bn - 1) / p.bn); };
  while (p.bn > 64 && units() < kPlanSms) p.bn /= 2;
  p.S = 1;
  const int64_t u = std::max<int64_t>(1, units());
  // pieces of at least 512 (FP8: 1024) of the reduction, partial sums within
  // the workspace's bound
  const int64_t step = kind == kMmFp8 ? 1024 : 512;
  const int64_t outs = (wg ? (int64_t)G * N : (int64_t)R) * cols;
  if (u < kPlanSms && outs > 0)
    p.S = (int)std::max<int64_t>(1, std::min({kPlanSms / u, red / step, kPartBytes / (outs * 4), (int64_t)32}));
  return p;
}
int mm_splits(int kind, int R, int N, int K, int G) { return mm_plan(kind, R, N, K, G).S; }

// ---- host -------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
bool make_tmap(CUtensorMap* map, const void* base, int esize, int rank, const int64_t* dims, const int64_t* strides,
               const int* box) {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return (EncodeTiledFn) nullptr;
  }();
  if (!fn) return false;
  cuuint64_t d[5], s[5];
  cuuint32_t b[5], e[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    e[i] = 1;
    if (i + 1 < rank) s[i] = (cuuint64_t)strides[i] * esize;
  }
  return fn(map, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, rank,
            const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [G][rows][cols] with cols contiguous and the MMA's M / N axis: 64-row
// boxes. Where cols is a whole number of 64-wide chunks, the map has a chunk
// axis and one copy brings `chunks` of them, one after the other (a copy
// costs its issuer more than its bytes); else a copy a chunk (a chunk axis
// would read past the last row's end). Returns the chunks a copy takes.
static int make_mn(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int64_t G, int64_t gs,
                   int chunks) {
  if (G == 1) gs = ld;      // never stepped over
  if (cols % 64 == 0 && chunks > 1) {
    const int64_t dims[4] = {64, rows, cols / 64, G}, strides[3] = {ld, 64, gs};
    const int box[4] = {64, kGK, chunks, 1};
    return make_tmap(map, base, 2, 4, dims, strides, box) ? chunks : 0;
  }
  const int64_t dims[4] = {cols, rows, 1, G}, strides[3] = {ld, ld, gs};
  const int box[4] = {64, kGK, 1, 1};
  return make_tmap(map, base, 2, 4, dims, strides, box) ? 1 : 0;
}

template <int MODE, int BN>
static cudaError_t launch_g(GArgs g, cudaStream_t st) {
  using C = GCfg<BN>;
  const MmArgs& m = g.m;
  constexpr bool kWg = MODE == kWgradMN;
  GMaps maps;
  const int64_t rows = std::max(m.R, 1);
  if (kWg) {
    // without rows nothing is copied, and the maps only need an aligned address
    const void* a = m.R > 0 ? m.a : m.status;
    const void* b = m.R > 0 ? m.b : m.status;
    g.a_chunks = make_mn(&maps.a[0], a, rows, m.N, m.lda, 1, 0, kGM / 64);
    g.b_chunks = make_mn(&maps.b, b, rows, m.K, m.ldb, 1, 0, BN / 64);
    if (!g.a_chunks || !g.b_chunks) return cudaErrorInvalidValue;
    g.m_tiles = (m.N + kGM - 1) / kGM;
    g.n_tiles = (m.K + BN - 1) / BN;
  } else {
    for (int i = 0; i < 4; ++i) {
      const int64_t dims[2] = {m.K, rows}, strides[1] = {m.lda};
      const int box[2] = {kGK, 16 << i};
      if (!make_tmap(&maps.a[i], m.a, 2, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (MODE == kRowsNT) {
      const int64_t dims[3] = {m.K, m.N, m.G}, strides[2] = {m.ldb, m.G > 1 ? m.bg : m.ldb};
      const int box[3] = {kGK, BN, 1};
      if (!make_tmap(&maps.b, m.b, 2, 3, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
      g.b_chunks = make_mn(&maps.b, m.b, m.K, m.N, m.ldb, m.G, m.bg, BN / 64);
      if (!g.b_chunks) return cudaErrorInvalidValue;
    }
    g.n_tiles = (m.N + BN - 1) / BN;
  }
  if (!units_fit(m, kWg ? (int64_t)m.G * g.m_tiles : m.R / kGM, g.n_tiles)) return cudaErrorInvalidValue;
  static std::atomic<bool> done[kMaxDevices] = {};
  cudaError_t e = set_smem_once((const void*)k_gemm16<MODE, BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_pdl(k_gemm16<MODE, BN>, dim3(device_sms()), dim3(kGThreads), C::kSmem, st, g, maps);
  if (e != cudaSuccess || m.S == 1) return e;
  return launch_mm_join(m, kWg, st);
}

template <int MODE>
static cudaError_t launch_bn(const GArgs& g, int bn, cudaStream_t st) {
  return bn == 256 ? launch_g<MODE, 256>(g, st) : bn == 128 ? launch_g<MODE, 128>(g, st) : launch_g<MODE, 64>(g, st);
}

cudaError_t launch_mm16(const MmArgs& a, bool wgrad, cudaStream_t st) {
  GArgs g = {};
  g.m = a;
  const int bn = mm_plan(wgrad ? kMmWgrad : kMmRows, a.R, a.N, a.K, a.G).bn;
  if (wgrad) return launch_bn<kWgradMN>(g, bn, st);
  return a.trans_b ? launch_bn<kRowsNN>(g, bn, st) : launch_bn<kRowsNT>(g, bn, st);
}

}  // namespace moe
