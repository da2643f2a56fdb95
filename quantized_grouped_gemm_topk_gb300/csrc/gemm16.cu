// Products grouped by expert with ragged sizes, bf16 or f16, on the
// 5th-generation tensor cores (tcgen05.mma kind::f16, operands in shared
// memory, fp32 accumulators in tensor memory). D[M][N] of a tile is
//
//   kRowsNT   out^T = W_e x^T    M features of W (K-major), N token rows of x
//   kRowsNN   out^T = W_e^T x^T  the same with W's feature axis contiguous (the
//             gradient of the rows with the forward's weights, no transpose)
//   kWgradMN  dW_e = dy^T x      M features of dy, N features of x, both
//             contiguous; the reduction runs over the group's rows
//
// The weights are the MMA's M side, so the ragged side is N: an instruction's
// N is the tile's real rows rounded up to 32, and a group of 300 rows costs
// 300, not the next multiple of 128 or 256; a decode step of a few rows costs
// little next to its weights' bytes.
//
// Bound: the tensor pipe at training sizes, the weights' bytes at decode
// sizes. What an SM can take in from L2 (64 bytes a cycle, measured: 48 KB
// took 745 cycles whatever else was changed) is less than a 128 x 256
// tile on one SM wants (48 KB per 512 cycles of MMA). So where there is work
// for it a pair of SMs (cta_group::2) multiplies a 256 x 256 tile together:
// 32 KB for each. Tiles of one SM (128 x up to 256) serve few tiles and few
// rows. Stages of 128 of the reduction in a ring that fills the shared memory,
// filled by tensor copies with the 128-byte swizzle. Ragged edges cost
// no branch in the main loop: rows of a tile that belong to the next group
// only reach accumulator columns that are not stored; columns and the K tail
// read as zeros (the tensor maps end at N and K); the weight gradient's last
// rows are cleared in shared memory, both operands (a NaN of the next group
// times zero would be NaN).
//
// Roles (a CTA an SM, persistent over the units): warp 0 copies B, warp 2
// copies A (two issuers: a copy costs its thread some hundred cycles), warp 1
// issues the MMAs (in a pair the first CTA's, whose barriers all copies of the
// pair report to), warps 4-7 and 8-11 are epilogues
// that alternate between tiles and the two accumulators, so a tile's stores
// overlap the next one's MMAs; warp 3 clears rows outside every group (weight
// gradient: those behind a group's last rows, in shared memory).
// Every wait is bounded; a CTA whose wait runs out sets MOE_DEV_TIMEOUT, waits
// for its copies and MMAs in flight, frees tensor memory and returns.
// Measured, bf16, in a burst and sustained (at the power limit, where the clock
// falls): 8192^3 NT 621 us (1.77 PFLOP/s) and 702, NN 634 and 708, weight gradient
// 632 and 706; 65536 rows in 128 groups x 5760 x 2880 1.47 ms (1.47 PFLOP/s, tensor
// pipe 68 % busy) and 1.67 (1.30); 30011 rows in 64 groups, 2880 x 2880 weight
// gradients 432 us and 465; 8 rows of 8 experts x 4096 x 7168 76 us (6.2 TB/s of
// weights).
#include "groups.cuh"
#include "tc.cuh"

namespace moe {

enum { kRowsNT = 0, kRowsNN = 1, kWgradMN = 2 };

// Reduction a stage: two halves of one 128-byte swizzle row each, which land
// behind one barrier and are freed one by one. The thread that issues the MMAs
// spends some 270 cycles a stage besides the MMAs themselves; with one half a
// stage that was the bound of tiles narrower than 256 (about 570 cycles a stage
// whatever their width).
constexpr int kGH = 64;
constexpr int kGK = 2 * kGH;
constexpr int kGN = 256;              // widest tile
constexpr int kGThreads = 384;
constexpr int kGChunk = 64 * kGH * 2; // bytes of 64 M / N elements of an MN-contiguous half
constexpr int kGABytes = kGM * kGH * 2;   // of a half
constexpr int kGHeadBars = 512;       // barriers and scratch, in front of the group tables
constexpr int kGMaxStages = 6;
constexpr int kGSmem = 227 * 1024;

constexpr int kGBoxes = 5;            // K-major B: boxes of 16 << i rows
struct GMaps {
  CUtensorMap a;
  CUtensorMap b[kGBoxes];             // MN-contiguous B: b[0]
};
struct GArgs {
  MmArgs m;
  int bn;               // widest N of a tile
  int stages;           // of the ring, each 2 (kGABytes + b_bytes)
  int b_bytes;          // of B's half
  int head;             // bytes in front of the ring
  int m_tiles;          // tiles of 128 CG features
  int n_tiles;          // weight gradient: bn-wide column tiles
  int a_chunks, b_chunks;   // MN-contiguous operands: 64-wide chunks a copy takes (1: one copy a chunk)
};

struct GTile {
  int e;
  int m0;               // first feature (row of D)
  int c0, nc, N;        // first token row (weight gradient: column), real ones, the MMA's N
  int k0, k1, red;      // stages [k0, k1) of the reduction's `red`
  int piece;
};

template <int MODE, int CG>
__device__ __forceinline__ void g_tile(const GArgs& g, const int32_t* off, const int32_t* uoff, int u, GTile& w) {
  const MmArgs& m = g.m;
  const int t = m.S == 1 ? u : u / m.S;
  w.piece = u - t * m.S;
  if (MODE == kWgradMN) {
    // units of a group: row tiles, then column tiles innermost
    const int ui = t / g.n_tiles;
    w.c0 = (t - ui * g.n_tiles) * g.bn;
    w.nc = min(g.bn, m.K - w.c0);
    w.N = g.bn;
    w.e = ui / g.m_tiles;
    w.m0 = (ui - w.e * g.m_tiles) * (kGM * CG);
    w.red = off[w.e + 1] - off[w.e];
  } else {
    // token tiles of a group, feature tiles innermost
    const int ui = t / g.m_tiles;
    w.m0 = (t - ui * g.m_tiles) * (kGM * CG);
    w.e = group_of_unit(uoff, m.G, ui);
    const int cnt = off[w.e + 1] - off[w.e], nt = uoff[w.e + 1] - uoff[w.e];
    // the group's rows in equal tiles, of a multiple of 32 each
    const int wide = (((cnt + nt - 1) / nt) + 31) & ~31;
    const int r = (ui - uoff[w.e]) * wide;
    w.c0 = off[w.e] + r;
    w.nc = min(wide, cnt - r);
    w.N = (w.nc + 31) & ~31;
    w.red = m.K;
  }
  const int nk = (w.red + kGK - 1) / kGK;
  w.k0 = m.S == 1 ? 0 : (int)((int64_t)nk * w.piece / m.S);
  w.k1 = m.S == 1 ? nk : (int)((int64_t)nk * (w.piece + 1) / m.S);
}

// A copy of K-major token rows covers 16 << i of them, the fewest that hold
// the tile's; what lies behind them in the stage only reaches columns that
// are not stored.
__device__ __forceinline__ int g_box(int rows) {
  return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 ? 3 : 4;
}

// The copies of a stage, by shared-memory addresses: into this CTA's memory,
// reported to `bar` (one SM: its own barrier; a pair: one of either CTA).
template <int CG>
__device__ __forceinline__ void g_copy2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (CG == 2) tc::tma_load_2d_pair(dst, map, x, y, bar);
  else tc::tma_load_2d_at(dst, map, x, y, bar);
}
template <int CG>
__device__ __forceinline__ void g_copy3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (CG == 2) tc::tma_load_3d_pair(dst, map, x, y, z, bar);
  else tc::tma_load_3d_at(dst, map, x, y, z, bar);
}
// An MN-contiguous operand: `chunks` chunks of 64 columns from column c0, rows
// row0 .. row0 + 63 of matrix z; one copy where the map has a chunk axis.
template <int CG>
__device__ __forceinline__ void g_copy_mn(uint32_t dst, const CUtensorMap* map, int c0, int row0, int z, int chunks,
                                          bool one, uint32_t bar) {
  const int n = one ? 1 : chunks;
  for (int c = 0; c < n; ++c) {
    const int x = one ? 0 : c0 + 64 * c, ch = one ? c0 / 64 : 0;
    if (CG == 2) tc::tma_load_4d_pair(dst + c * kGChunk, map, x, row0, ch, z, bar);
    else tc::tma_load_4d_at(dst + c * kGChunk, map, x, row0, ch, z, bar);
  }
}

template <int CG>
__device__ __forceinline__ void g_commit(uint32_t bar) {
  if (CG == 2) tc::bar_commit_pair(bar);
  else tc::bar_commit(bar);
}

// Whether a stage of the weight gradient ends inside an MMA's K of 16: the
// group's last rows, `left` of them; the rows behind are cleared in shared
// memory by each CTA before the MMAs read them.
__device__ __forceinline__ bool g_tail(int left) { return left < kGK && (left & 15); }

// 32 token rows (n of them real) of the lane's feature: out[row][f], f =
// f0 + lane < F. 16-bit outputs: two lanes exchange so that each stores two
// neighbouring features of one row (`pairs`: 4-byte stores are aligned).
template <typename E>
__device__ __forceinline__ void store_tokens16(uint16_t* out, int64_t ld, const uint32_t (&v)[32], int n, int lane,
                                               int f0, int F, bool pairs) {
  if (pairs && f0 + 32 <= F) {
    const bool odd = lane & 1;
    uint16_t* p = out + f0 + (lane & ~1) + (odd ? ld : 0);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint32_t other = __shfl_xor_sync(kFull, odd ? v[i] : v[i + 1], 1);
      const uint32_t w = odd ? E::from2(__uint_as_float(other), __uint_as_float(v[i + 1]))
                             : E::from2(__uint_as_float(v[i]), __uint_as_float(other));
      if (i + (odd ? 1 : 0) < n) *reinterpret_cast<uint32_t*>(p + i * ld) = w;
    }
  } else if (f0 + lane < F) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) out[i * ld + f0 + lane] = E::from(__uint_as_float(v[i]));
  }
}

template <int MODE, int CG>
__global__ void __launch_bounds__(kGThreads, 1) k_gemm16(const GArgs g, const __grid_constant__ GMaps maps) {
  constexpr bool kWg = MODE == kWgradMN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int stages = g.stages, b_bytes = g.b_bytes;
  uint8_t* sa = base + g.head;
  uint8_t* sb = sa + stages * 2 * kGABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* pfull = full + kGMaxStages;         // weight gradient: the rows of a tail stage are cleared
  uint64_t* empty = pfull + kGMaxStages;
  uint64_t* accfull = empty + 2 * kGMaxStages;    // empty: of each half
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint64_t* tgo = drain + 1;                    // weight gradient: a tail stage has landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tgo + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tmp = reinterpret_cast<int*>(tmem_slot + 2);
  int32_t* off = reinterpret_cast<int32_t*>(base + kGHeadBars);
  int32_t* uoff = off + g.m.G + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MmArgs& m = g.m;
  const int rank = CG == 2 ? (int)tc::cluster_rank() : 0;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      tc::mbar_init(&full[i], 2);       // one arrival (with its bytes) from each copying warp
      tc::mbar_init(&pfull[i], CG);
      tc::mbar_init(&empty[2 * i], 1);
      tc::mbar_init(&empty[2 * i + 1], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], 1);
      tc::mbar_init(&accempty[i], 4 * CG);   // one per epilogue warp of the tile, of both CTAs
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init(tgo, 1);
    *abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    if (CG == 2) tc::tmem_alloc_pair(tmem_slot, 512);
    else tc::tmem_alloc(tmem_slot, 512);
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&maps.a);
    for (int i = 0; i < (kWg ? 1 : kGBoxes); ++i) tc::prefetch_tmap(&maps.b[i]);
  }
  pdl_enter();
  build_groups<kGThreads>(m.offsets, m.G, m.R, off, uoff, tmp, m.status,
                          [&](int c) { return kWg ? g.m_tiles : (c + g.bn - 1) / g.bn; });
  tc::fence_before_sync();
  __syncthreads();
  // the peer's barriers are initialised before anything reaches them
  if constexpr (CG == 2) tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int U = uoff[m.G] * (kWg ? g.n_tiles : g.m_tiles) * m.S;

  const uint32_t full_u = tc::smem_u32(full), pfull_u = tc::smem_u32(pfull), empty_u = tc::smem_u32(empty);
  const uint32_t sa_u = tc::smem_u32(sa), sb_u = tc::smem_u32(sb);
  if (warp == 0 || warp == 2) {
    // ---------------- copies: warp 0 B, warp 2 A ----------------
    if (lane == 0) {
      const bool isb = warp == 0;
      const uint32_t dst0 = isb ? sb_u : sa_u, half_bytes = isb ? b_bytes : kGABytes;
      // both CTAs' copies report to the first one's barriers, which expect them
      // all; those of a tail stage, where each CTA has rows to clear first, to
      // their own CTA's
      const uint32_t lead_u = CG == 2 ? tc::peer_smem(full, 0) : full_u;
      int slot = 0;
      uint32_t phase = 1;          // of empty: the ring starts free
      uint32_t issued = 0;
      bool ok = true;
      for (int u = first; ok && u < U; u += stride) {
        GTile w;
        g_tile<MODE, CG>(g, off, uoff, u, w);
        const int half = w.N / CG;                    // B rows of this CTA
        const int c0 = w.c0 + rank * half, m0 = w.m0 + rank * kGM;
        const int bi = g_box(half);
        const uint32_t bytes = !isb ? kGABytes : kWg ? (uint32_t)(half / 64 * kGChunk) : (uint32_t)(kGH * 2 * (16 << bi));
        const CUtensorMap* map = isb ? (kWg ? &maps.b[0] : &maps.b[bi]) : &maps.a;
        const int r0 = kWg ? off[w.e] : 0;
        for (int kb = w.k0; kb < w.k1; ++kb) {
          const int k = kb * kGK;
          const bool own = CG == 1 || (kWg && g_tail(w.red - k));
          const uint32_t bar = (own ? full_u : lead_u) + 8 * slot;
          uint32_t dst = dst0 + slot * 2 * half_bytes;
          const int halves = w.red - k > kGH ? 2 : 1;
          // each half is refilled as soon as its own MMAs are done
          for (int s = 0; s < 2; ++s, dst += half_bytes) {
            if (!tc::bar_wait(empty_u + 16 * slot + 8 * s, phase, abort)) { ok = false; break; }
            if (s == 0 && (own || rank == 0))
              tc::bar_arrive_expect_tx(full_u + 8 * slot, (own ? bytes : CG * bytes) * halves);
            if (s == halves) break;
            const int ks = k + s * kGH;
            if (isb) {
              if (kWg) g_copy_mn<CG>(dst, map, c0, r0 + ks, 0, half / 64, g.b_chunks > 1, bar);
              else g_copy2<CG>(dst, map, ks, c0, bar);
            } else {
              if (MODE == kRowsNT) g_copy3<CG>(dst, map, ks, m0, w.e, bar);
              else g_copy_mn<CG>(dst, map, m0, kWg ? r0 + ks : ks, kWg ? 0 : w.e, kGM / 64, g.a_chunks > 1, bar);
            }
            if (s == 0) ++issued;        // counted as soon as a copy of the stage is in flight
          }
          if (!ok) break;
          if (++slot == stages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok || *abort) {
        // wind-down: wait (bounded, ignoring the abort flag) for the copies
        // this thread still has in flight. A slot's barrier completes only
        // when the other copying warp arrived too; it may have stopped
        // earlier (and the second CTA of a pair reports elsewhere), so the
        // wait's limit is what ends this then.
        volatile int never = 0;
        const uint32_t n = issued < (uint32_t)stages ? issued : (uint32_t)stages;
        for (uint32_t k = 0; k < n; ++k) {
          const uint32_t i2 = issued - 1 - k;
          tc::mbar_wait(&full[i2 % stages], (i2 / stages) & 1, &never, 100000000ll);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    // One thread, whose loop bounds the whole when it is longer than the MMAs:
    // addresses, descriptors and parities are carried along, not computed.
    if (lane == 0 && rank == 0) {
      constexpr uint32_t sta = MODE != kRowsNT ? 2048 / 16 : 32 / 16, stb = kWg ? 2048 / 16 : 32 / 16;
      const uint64_t ad0 = MODE != kRowsNT ? tc::smem_desc_mn_sw128(sa_u, kGChunk) : tc::smem_desc_sw128(sa_u);
      const uint64_t bd0 = kWg ? tc::smem_desc_mn_sw128(sb_u, kGChunk) : tc::smem_desc_sw128(sb_u);
      const uint32_t a_hi = (uint32_t)(ad0 >> 32), b_hi = (uint32_t)(bd0 >> 32), a_half = kGABytes / 16, b_half = b_bytes / 16;
      uint32_t ad = (uint32_t)ad0, bd = (uint32_t)bd0;
      int slot = 0;
      uint32_t phase = 0, tails = 0;     // tails: parity, by slot, of pfull
      uint32_t tcount = 0;
      bool ok = true, ready = false;     // ready: the next stage is known to have landed
      for (int u = first; ok && u < U; u += stride, ++tcount) {
        GTile w;
        g_tile<MODE, CG>(g, off, uoff, u, w);
        const int d = tcount & 1;
        if (!tc::mbar_wait(&accempty[d], ((tcount >> 1) & 1) ^ 1, abort)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t dt = tmem + d * kGN;
        const uint32_t idesc = tc::idesc_16bit(kGM * CG, w.N, m.dtype == MOE_DT_BF16, MODE != kRowsNT, kWg);
        uint32_t acc = 0;
        int left = w.red - w.k0 * kGK;
        for (int n = w.k1 - w.k0; n > 0; --n, left -= kGK) {
          if (!ready && !tc::bar_wait(full_u + 8 * slot, phase, abort)) { ok = false; break; }
          const uint32_t done = empty_u + 16 * slot, a_now = ad, b_now = bd;
          const int slot_now = slot;
          ad += 2 * a_half;
          bd += 2 * b_half;
          if (++slot == stages) {
            slot = 0;
            phase ^= 1;
            ad = (uint32_t)ad0;
            bd = (uint32_t)bd0;
          }
          // asked now, so that the answer's latency passes behind the MMAs' issue
          ready = tc::bar_test(full_u + 8 * slot, phase);
          if (kWg && g_tail(left)) {
            // warp 3 (of both CTAs) clears the rows of the next group. No step
            // of the stage is issued before: that the second CTA's copies have
            // landed is only known from its arrival
            tc::mbar_arrive(tgo);
            if (!tc::bar_wait(pfull_u + 8 * slot_now, (tails >> slot_now) & 1, abort)) { ok = false; break; }
            tails ^= 1u << slot_now;
          }
          tc::fence_after_sync();
          // a step of K = 16: 32 bytes along a K-major row, two 8-row atoms otherwise
          if (left > kGK - 16) {
            tc::mma_f16_x4<CG>(dt, a_now, a_hi, sta, b_now, b_hi, stb, idesc, acc);
            g_commit<CG>(done);
            tc::mma_f16_x4<CG>(dt, a_now + a_half, a_hi, sta, b_now + b_half, b_hi, stb, idesc, 1u);
          } else {
            const int steps = (left + 15) / 16;
            for (int j = 0; j < steps; ++j) {
              const uint32_t al = a_now + (j >= 4 ? a_half : 0u) + sta * (j & 3);
              const uint32_t bl = b_now + (j >= 4 ? b_half : 0u) + stb * (j & 3);
              const uint64_t da = ((uint64_t)a_hi << 32) | al, db = ((uint64_t)b_hi << 32) | bl;
              if constexpr (CG == 2) tc::mma_f16_ss_pair(dt, da, db, idesc, j ? 1u : acc);
              else tc::mma_f16_ss(dt, da, db, idesc, j ? 1u : acc);
            }
            g_commit<CG>(done);
          }
          g_commit<CG>(done + 8);
          acc = 1;
        }
        if (!ok) break;
        if constexpr (CG == 2) tc::mma_commit_pair(&accfull[d]);
        else tc::mma_commit(&accfull[d]);
      }
      // every MMA of this thread has completed once `drain` fires
      if constexpr (CG == 2) tc::mma_commit_pair(drain);
      else tc::mma_commit(drain);
      volatile int never = 0;
      tc::mbar_wait(drain, 0, &never, 400000000ll);
    }
    __syncwarp();
  } else if (warp == 3) {
    if (!kWg) {
      clear_rows_outside(m, off, lane);
    } else {
      // ---------------- tail stages ----------------
      // Rows behind a group's last ones: cleared up to the MMA's K, a 128-byte
      // line per row and chunk (the swizzle permutes within a line). This warp
      // is told of a landed tail stage (`tgo`, by the MMA thread; in the second
      // CTA of a pair, whose barriers only tail stages use, by the copies): it
      // would miss phases of a barrier that does not wait for it.
      int slot = 0;
      uint32_t told = 0, tails = 0;
      for (int u = first; u < U; u += stride) {
        GTile w;
        g_tile<MODE, CG>(g, off, uoff, u, w);
        const int n = w.k1 - w.k0, left = w.red - (w.k1 - 1) * kGK;
        const int at = (slot + n + stages - 1) % stages;     // the piece's last stage
        slot = (slot + n) % stages;
        if (n <= 0 || !g_tail(left)) continue;
        const bool got = rank == 0 ? tc::mbar_wait(tgo, told, abort)
                                   : tc::mbar_wait(&full[at], (tails >> at) & 1, abort);
        if (!__all_sync(kFull, got)) break;
        told ^= 1;
        tails ^= 1u << at;
        // eight lanes a line, four lines at a time: the MMAs wait for this (with
        // a division for each store 64 groups of 385 rows x 2880 x 2880 took 499 us,
        // now 410, and of 470 rows 492, now 434)
        const int bad = 16 - (left & 15), at0 = (left % kGH + (lane >> 3)) * 128 + (lane & 7) * 16;
        auto clear = [&](uint8_t* p, int chunks) {
          for (int c = 0; c < chunks; ++c, p += kGChunk)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
              if (r + (lane >> 3) < bad) *reinterpret_cast<uint4*>(p + r * 128) = make_uint4(0u, 0u, 0u, 0u);
        };
        // in the half that `left` ends in
        clear(sa + (2 * at + left / kGH) * kGABytes + at0, kGM / 64);
        clear(sb + (2 * at + left / kGH) * b_bytes + at0, w.N / CG / 64);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (CG == 2 && rank != 0) tc::mbar_arrive_peer(tc::peer_smem(&pfull[at], 0));
          else tc::mbar_arrive(&pfull[at]);
        }
        __syncwarp();
      }
    }
  } else {
    // ---------------- epilogue ----------------
    const int wg = (warp - 4) >> 2, q = warp & 3;
    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + wg * kGN;
    const int cols = kWg ? m.K : m.N;               // of a row of out
    const int dt = m.S > 1 ? MOE_DT_F32 : m.out_dtype;
    const int esize = dt == MOE_DT_F32 ? 4 : 2;
    const int64_t ld = m.S > 1 ? cols : m.ldo;
    uint8_t* obase = reinterpret_cast<uint8_t*>(m.S > 1 ? (void*)m.part : m.out);
    const int64_t og = m.S > 1 ? (int64_t)m.N * m.K : m.og;
    const int64_t os = kWg ? (int64_t)m.G * m.N * m.K : (int64_t)m.R * m.N;      // a piece's partial sums
    const bool vec = ((uintptr_t)obase & 15) == 0 && (ld * esize) % 16 == 0 && (og * esize) % 16 == 0 &&
                     (m.S == 1 || (os * 4) % 16 == 0);
    const bool pairs = ((uintptr_t)obase & 3) == 0 && ld % 2 == 0;
    uint32_t tcount = 0, mine = 0;
    for (int u = first; u < U; u += stride, ++tcount) {
      if ((int)(tcount & 1) != wg) continue;
      GTile w;
      g_tile<MODE, CG>(g, off, uoff, u, w);
      const bool got = tc::mbar_wait(&accfull[wg], mine & 1, abort);
      if (!__all_sync(kFull, got)) break;
      tc::fence_after_sync();
      const int f0 = w.m0 + rank * kGM + q * 32;    // the warp's first feature
      if constexpr (kWg) {
        // 64 columns at a time: a row's 128 bytes (16-bit), exchanged between
        // the lanes before they are stored
        const int rows = m.N - f0;
        const int64_t at0 = w.e * og + (int64_t)f0 * ld + w.c0 + (m.S > 1 ? w.piece * os : 0);
        for (int c = 0; c < w.nc; c += 64) {
          uint32_t v[64];
          if (w.k1 > w.k0) {
            tc::tmem_ld32(acc + c, reinterpret_cast<uint32_t(&)[32]>(v[0]));
            tc::tmem_ld32(acc + c + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]));
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = 0u;       // no rows to sum over
          }
          if (vec && c + 64 <= w.nc) {
            float f[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) f[i] = __uint_as_float(v[i]);
            store_block<64>(obase + (at0 + c) * esize, ld * esize, f, rows, lane, dt);
          } else if (lane < rows) {
            store_cols<64>(obase + (at0 + lane * ld + c) * esize, v, w.nc - c, dt, vec);
          }
          __syncwarp();
        }
      } else {
        for (int c = 0; c < w.nc; c += 32) {
          uint32_t v[32];
          if (w.k1 > w.k0) {
            tc::tmem_ld32(acc + c, v);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          const int64_t at = (int64_t)(w.c0 + c) * ld + (m.S > 1 ? w.piece * os : 0);
          const int n = w.nc - c;
          if (dt == MOE_DT_F32) {
            float* p = reinterpret_cast<float*>(obase) + at + f0 + lane;
            if (f0 + lane < m.N) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < n) p[i * ld] = __uint_as_float(v[i]);
            }
          } else if (dt == MOE_DT_F16) {
            store_tokens16<F16>(reinterpret_cast<uint16_t*>(obase) + at, ld, v, n, lane, f0, m.N, pairs);
          } else {
            store_tokens16<Bf16>(reinterpret_cast<uint16_t*>(obase) + at, ld, v, n, lane, f0, m.N, pairs);
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0) tc::mbar_arrive_peer(tc::peer_smem(&accempty[wg], 0));
        else tc::mbar_arrive(&accempty[wg]);
      }
      ++mine;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  // neither CTA of a pair leaves while the other's MMAs read its memory or its
  // arrivals are on their way
  if constexpr (CG == 2) tc::cluster_sync();
  if (threadIdx.x == 0 && *abort) set_status(m.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    if (CG == 2) tc::tmem_dealloc_pair(tmem, 512);
    else tc::tmem_dealloc(tmem, 512);
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
constexpr int64_t kStep16 = 512, kStepFp8 = 1024;     // least reduction of a piece

static int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

MmPlan mm_plan(int kind, int R, int N, int K, int G) {
  const bool wg = kind == kMmWgrad;
  MmPlan p = {1, 256, 1};
  // tiles of `b` rows: at least one for every group that can have rows
  auto row_tiles = [&](int b) { return std::max<int64_t>(tiles(R, b), std::min(G, R)); };
  auto count = [&](int cg, int bn) {
    if (kind == kMmFp8) return row_tiles(kGM) * tiles(N, bn);
    return wg ? G * tiles(N, kGM * cg) * tiles(K, bn) : row_tiles(bn) * tiles(N, kGM * cg);
  };
  if (kind != kMmFp8) {
    // Pairs of SMs where there is a tile for each of them, except at a few
    // rows a group, which stream weights. 4096 x 7168 weights, 32 groups: 256
    // rows 276 us with single SMs, 281 with pairs; 1024 rows 283 and 280; 2048
    // rows 324 and 301. One group, 8192^3: 755 and 615.
    p.cg = count(2, 256) >= kPlanSms / 2 && (wg || R >= 64ll * std::min(G, R)) ? 2 : 1;
    // Few rows a group: narrow tiles, whose stages are small, so that more of
    // them are in flight (the same weights: 8 rows 76 us, 91 with wide tiles;
    // 1024 rows 283 and 319).
    if (!wg && R <= 32ll * std::min(G, R)) p.bn = R <= 8ll * std::min(G, R) ? 32 : 64;
  }
  if (p.cg == 1 && p.bn > 64) {
    // The width that takes the least time: rounds of tiles over the SMs times
    // a stage's bytes, 128 + bn rows of an operand, which bound it. Against
    // the widest with a tile for every SM: FP8 1024 x 2048 x 4096 18.4 us (28.7),
    // 512 x 7168 x 4096 24 (32), 1500 x 4096 x 2048 27 (26); bf16 1024 x 2880 x
    // 2880 24 (28), 1500 x 2048 x 7168 48 (58). Against the widest of all: FP8
    // 3 x 7168 x 2048 10.6 us (13.3).
    int64_t least = INT64_MAX;
    for (int bn = p.bn; bn >= 64; bn /= 2) {
      const int64_t cost = tiles(count(1, bn), kPlanSms) * (kGM + bn);
      if (cost <= least) {
        least = cost;
        p.bn = bn;
      }
    }
  }
  const int64_t units = count(p.cg, p.bn);
  // Too few tiles: pieces of at least kStep16 (kStepFp8) of the reduction, partial
  // sums within the workspace's bound (bf16 64 x 2880 x 2880 14.8 us, 20.7 in
  // one piece).
  const int64_t red = wg ? tiles(R, G) : K, step = kind == kMmFp8 ? kStepFp8 : kStep16;
  const int64_t outs = wg ? (int64_t)G * N * K : (int64_t)R * N;
  if (p.cg == 1 && units > 0 && units < kPlanSms && outs > 0)
    p.S = (int)std::max<int64_t>(1, std::min({kPlanSms / units, red / step, kPartBytes / (outs * 4), (int64_t)32}));
  return p;
}
int mm_splits(int kind, int R, int N, int K, int G) { return mm_plan(kind, R, N, K, G).S; }
int64_t mm_part_bytes(int kind, int R, int N, int K, int G) {
  if (kind == kMmWgrad) {       // the pieces only grow in number with the rows
    const int S = mm_splits(kind, R, N, K, G);
    return S > 1 ? (int64_t)G * N * K * 4 * S : 0;
  }
  // Few rows are cut into more pieces than many, so the need of R rows says
  // nothing about fewer. Any of them: at most this many pieces, and together at
  // most kPlanSms tiles of 128 x 256 outputs.
  const int64_t most = std::min({(int64_t)32, K / (kind == kMmFp8 ? kStepFp8 : kStep16),
                                 kPlanSms / tiles(N, kind == kMmFp8 ? 256 : kGM)});
  return most > 1 ? std::min<int64_t>((int64_t)R * N * 4 * most, (int64_t)kPlanSms * kGM * 256 * 4) : 0;
}

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
// would read past the last row's end). Returns the chunks a copy takes, 0 if
// the map cannot be made.
static int make_mn(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int64_t G, int64_t gs,
                   int chunks) {
  if (G == 1) gs = ld;      // never stepped over
  if (cols % 64 == 0 && chunks > 1) {
    const int64_t dims[4] = {64, rows, cols / 64, G}, strides[3] = {ld, 64, gs};
    const int box[4] = {64, kGH, chunks, 1};
    return make_tmap(map, base, 2, 4, dims, strides, box) ? chunks : 0;
  }
  const int64_t dims[4] = {cols, rows, 1, G}, strides[3] = {ld, ld, gs};
  const int box[4] = {64, kGH, 1, 1};
  return make_tmap(map, base, 2, 4, dims, strides, box) ? 1 : 0;
}

template <int MODE, int CG>
static cudaError_t launch_g(GArgs g, cudaStream_t st) {
  const MmArgs& m = g.m;
  constexpr bool kWg = MODE == kWgradMN;
  // as many stages as fit: the ring's round trip (copy, MMAs, release) is long
  g.b_bytes = g.bn / CG * kGH * 2;
  g.head = (kGHeadBars + 2 * 4 * (m.G + 1) + 1023) / 1024 * 1024;
  const int stage = 2 * (kGABytes + g.b_bytes);
  g.stages = std::min(kGMaxStages, (kGSmem - 1024 - g.head) / stage);
  const int smem = 1024 + g.head + g.stages * stage;
  GMaps maps;
  const int64_t rows = std::max(m.R, 1);
  g.m_tiles = (int)tiles(m.N, kGM * CG);
  g.n_tiles = kWg ? (int)tiles(m.K, g.bn) : 1;
  if (kWg) {
    // without rows nothing is copied, and the maps only need an aligned address
    const void* a = m.R > 0 ? m.a : m.status;
    const void* b = m.R > 0 ? m.b : m.status;
    g.a_chunks = make_mn(&maps.a, a, rows, m.N, m.lda, 1, 0, kGM / 64);
    g.b_chunks = make_mn(&maps.b[0], b, rows, m.K, m.ldb, 1, 0, g.bn / CG / 64);
    if (!g.a_chunks || !g.b_chunks) return cudaErrorInvalidValue;
  } else {
    for (int i = 0; i < kGBoxes; ++i) {
      const int64_t dims[2] = {m.K, rows}, strides[1] = {m.lda};
      const int box[2] = {kGH, 16 << i};
      if (!make_tmap(&maps.b[i], m.a, 2, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (MODE == kRowsNT) {
      const int64_t dims[3] = {m.K, m.N, m.G}, strides[2] = {m.ldb, m.G > 1 ? m.bg : m.ldb};
      const int box[3] = {kGH, kGM, 1};
      if (!make_tmap(&maps.a, m.b, 2, 3, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
      g.a_chunks = make_mn(&maps.a, m.b, m.K, m.N, m.ldb, m.G, m.bg, kGM / 64);
      if (!g.a_chunks) return cudaErrorInvalidValue;
    }
  }
  if (!units_fit(m, kWg ? (int64_t)m.G * g.m_tiles : m.R / g.bn, kWg ? g.n_tiles : g.m_tiles))
    return cudaErrorInvalidValue;
  static std::atomic<bool> done[kMaxDevices] = {};
  cudaError_t e = set_smem_once((const void*)k_gemm16<MODE, CG>, kGSmem, done);
  if (e != cudaSuccess) return e;
  note_launch();
  if constexpr (CG == 1) {
    e = launch_pdl(k_gemm16<MODE, CG>, dim3(device_sms()), dim3(kGThreads), smem, st, g, maps);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // pairs that are resident at once, asked once per device
    static std::atomic<int> pairs[kMaxDevices] = {};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const bool slot = dev >= 0 && dev < kMaxDevices;
    int np = slot ? pairs[dev].load(std::memory_order_acquire) : 0;
    if (np <= 0) {
      cfg.gridDim = dim3(CG * (device_sms() / CG));
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&np, k_gemm16<MODE, CG>, &cfg) != cudaSuccess || np <= 0)
        np = std::max(1, device_sms() / CG);
      if (slot) pairs[dev].store(np, std::memory_order_release);
    }
    cfg.gridDim = dim3(CG * np);
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_gemm16<MODE, CG>, g, maps);
  }
  if (e != cudaSuccess || m.S == 1) return e;
  return launch_mm_join(m, kWg, st);
}

template <int MODE>
static cudaError_t launch_cg(const GArgs& g, int cg, cudaStream_t st) {
  return cg == 2 ? launch_g<MODE, 2>(g, st) : launch_g<MODE, 1>(g, st);
}

cudaError_t launch_mm16(const MmArgs& a, bool wgrad, cudaStream_t st) {
  GArgs g = {};
  g.m = a;
  const MmPlan p = mm_plan(wgrad ? kMmWgrad : kMmRows, a.R, a.N, a.K, a.G);
  g.bn = p.bn;
  if (wgrad) return launch_cg<kWgradMN>(g, p.cg, st);
  return a.trans_b ? launch_cg<kRowsNN>(g, p.cg, st) : launch_cg<kRowsNT>(g, p.cg, st);
}

}  // namespace moe
