// Products of 16-bit weights with a few rows, on the 5th-generation tensor
// cores, in one launch: the routed layer's both products with the activation and
// the combine between and behind them, or one dense product with its epilogue.
//
// Bound: the weights' bytes. Everything else is arranged around their stream.
//
// - Weights are the MMA's M side (128 features; gated: 64 gate and the matching
//   64 up features, which one tensor copy brings), the rows its N (16 to 256).
//   The first product multiplies every expert's weights with all the tokens:
//   up to 64 columns cost the tensor core no more than 16, and no gather is
//   needed. The epilogue reads the columns of the expert's own tokens; what the
//   others hold never leaves tensor memory, so a NaN stays with its token.
// - The work of a product is cut into equal shares of its stages, one to a CTA,
//   wherever the tiles end (few tiles over 152 SMs would leave up to half of
//   them idle in the last round). A tile that spans shares leaves fp32 partial
//   sums; the last CTA to finish one of its pieces adds them in order. No sum
//   depends on which CTA does what.
// - The second product's weights do not depend on the first one: their copies
//   run ahead into the ring while the CTA's B copies wait for all of the first
//   product's tiles, so the barrier between the products costs no stream time
//   as long as it is shorter than the ring (200 KB, 4.5 us).
// - CTAs claim their shares from a counter, all of the first product's before
//   any of the second's: a CTA that waits only waits for shares that running
//   CTAs hold, however many of the grid are resident.
//
// Roles: warp 0 claims and copies weights, warp 2 copies rows, warp 1 issues the
// MMAs, warps 4-7 are the epilogue (two accumulators, so that it overlaps the
// next tile's MMAs). Every wait is bounded; a CTA whose wait runs out sets
// MOE_DEV_TIMEOUT, waits for its copies and MMAs in flight, frees tensor memory
// and returns.
#include "few16.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kFM = 128;              // features a tile (MMA M)
constexpr int kFH = 64;               // reduction of a half stage: one 128-byte swizzle row
constexpr int kFK = 2 * kFH;
constexpr int kFThreads = 256;
constexpr int kFA = kFM * kFH * 2;    // bytes of A's half
constexpr int kFMaxStages = 8;
constexpr int kFBars = 512;           // barriers and scratch, in front of the tables
constexpr int kFSmem = 227 * 1024;
constexpr int kFCols = 8;             // columns the epilogue stages at a time
constexpr int kFQueue = 4;            // claimed shares in flight

struct FewMaps {
  CUtensorMap a[2];                   // weights: [G][halves][rows][K], box 64 x rows x halves
  CUtensorMap x;                      // rows of the (first) product, box 64 x N
  CUtensorMap y[4];                   // layer: rows of the second, boxes of 16, 32, 48, 64
};

// A product cut into shares.
struct Cut {
  int mt, nk, ng;                     // feature tiles, stages of the reduction, groups
  int P;                              // shares
  int64_t total;                      // stages
  __device__ __forceinline__ int64_t begin(int s) const { return total * s / P; }
  __device__ __forceinline__ int share_of(int64_t step) const { return (int)(((step + 1) * P - 1) / total); }
};
// A piece of a tile: stages [k0, k1) of tile (gi, j).
struct Piece {
  int gi, j, k0, k1;
  int64_t t0;                         // the tile's first stage
};
template <bool SECOND>
__device__ __forceinline__ void piece_at(const Cut& c, int64_t at, int64_t end, Piece& p) {
  const int64_t tile = at / c.nk;
  p.t0 = tile * c.nk;
  p.k0 = (int)(at - p.t0);
  p.k1 = (int)min((int64_t)c.nk, end - p.t0);
  if (SECOND) {                       // groups innermost: a share holds one feature tile's, by and large
    p.j = (int)(tile / c.ng);
    p.gi = (int)(tile - (int64_t)p.j * c.ng);
  } else {
    p.gi = (int)(tile / c.mt);
    p.j = (int)(tile - (int64_t)p.gi * c.mt);
  }
}

__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tma_weights(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}
// The epilogue's warps only.
__device__ __forceinline__ void epi_sync() { __syncwarp(); asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Whether `ok` holds for all of them: what one of them gives up, all do.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// Position of the lowest set bit, which is cleared.
__device__ __forceinline__ int next_bit(unsigned long long& m) {
  const int b = __ffsll((long long)m) - 1;
  m &= m - 1;
  return b;
}

template <typename E, bool LAYER>
__global__ void __launch_bounds__(kFThreads, 1) k_few16(const FewArgs g, const __grid_constant__ FewMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* empty = full + kFMaxStages;
  uint64_t* accfull = empty + kFMaxStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* qfull = accempty + 2;
  uint64_t* qempty = qfull + kFQueue;
  uint64_t* drain = qempty + kFQueue;
  int* queue = reinterpret_cast<int*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(queue + kFQueue);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tmp = reinterpret_cast<int*>(tmem_slot + 2);       // 2 + 2 * 8
  float* stage = reinterpret_cast<float*>(base + kFBars); // [kFCols][128]
  // layer's tables
  const int G = g.E + g.S, kp = g.k + g.S;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(base + kFBars + kFCols * kFM * 4);   // [G] tokens
  int* rowof = reinterpret_cast<int*>(mask + (LAYER ? G : 0));     // [G] first row of the group
  int* glist = rowof + (LAYER ? G : 0);                            // [ng] groups with tokens
  int* srow = glist + (LAYER ? min(G, g.R * kp) : 0);              // [T kp] row of a token's slot, -1: none
  float* wrow = reinterpret_cast<float*>(srow + (LAYER ? g.R * kp : 0));   // [rows] routing weight
  uint8_t* sa = base + g.head;
  uint8_t* sb = sa + g.stages * 2 * kFA;
  const int b_half = g.N * 128;                                    // bytes of B's half
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < g.stages; ++i) {
      tc::mbar_init(&full[i], 2);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], 1);
      tc::mbar_init(&accempty[i], 4);
    }
    for (int i = 0; i < kFQueue; ++i) {
      tc::mbar_init(&qfull[i], 1);
      tc::mbar_init(&qempty[i], 3);       // rows' copies, MMAs, epilogue
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.a[0]);
    tc::prefetch_tmap(&maps.x);
  }
  const uint32_t ncol = g.N <= 32 ? 32 : g.N <= 64 ? 64 : g.N <= 128 ? 128 : 256;     // of an accumulator
  if (warp == 1) tc::tmem_alloc(tmem_slot, 2 * ncol);
  if (LAYER)
    for (int i = tid; i < G; i += kFThreads) mask[i] = i >= g.E ? (g.R == 64 ? ~0ull : (1ull << g.R) - 1) : 0ull;
  pdl_enter();
  __syncthreads();

  Cut c1 = {g.mt1, g.nk1, 1, 1, 0}, c2 = {g.mt2, g.nk2, 0, 1, 0};
  if constexpr (LAYER) {
    // the tokens of every expert; an assignment of weight 0 is left out
    const int A = g.R * g.k;
    for (int a = tid; a < A; a += kFThreads) {
      const int e = g.ids[a];
      if (e < 0 || e >= g.E) {
        if (blockIdx.x == 0) set_status(g.status, MOE_DEV_BAD_EXPERT_ID);
      } else if (g.wts[a] != 0.f) {
        atomicOr(&mask[e], 1ull << (a / g.k));
      }
    }
    __syncthreads();
    // groups with tokens, and every group's first row: prefix sums over the groups
    const int per = (G + kFThreads - 1) / kFThreads, e0 = tid * per, e1 = min(G, e0 + per);
    int live = 0, rows = 0;
    for (int e = e0; e < e1; ++e) {
      live += mask[e] != 0;
      rows += __popcll(mask[e]);
    }
    int il = live, ir = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(kFull, il, o), b = __shfl_up_sync(kFull, ir, o);
      if (lane >= o) { il += a; ir += b; }
    }
    if (lane == 31) { tmp[2 + warp] = il; tmp[10 + warp] = ir; }
    __syncthreads();
    il -= live;
    ir -= rows;
    for (int w = 0; w < warp; ++w) { il += tmp[2 + w]; ir += tmp[10 + w]; }
    for (int e = e0; e < e1; ++e) {
      rowof[e] = ir;
      if (mask[e]) glist[il++] = e;
      ir += __popcll(mask[e]);
    }
    if (tid == kFThreads - 1) tmp[0] = il;
    __syncthreads();
    c1.ng = c2.ng = tmp[0];
    // rows and weights of the slots: a repeated id's weights add up, in slot order, at its first slot
    for (int a = tid; a < g.R * kp; a += kFThreads) {
      const int t = a / kp, j = a - t * kp;
      int row = -1;
      float w = 1.f;
      int e = g.E + j - g.k;
      bool first = true;
      if (j < g.k) {
        e = g.ids[t * g.k + j];
        first = e >= 0 && e < g.E && (mask[e] >> t & 1);
        if (first) {
          w = 0.f;
          for (int i = 0; i < g.k; ++i)
            if (g.ids[t * g.k + i] == e) {
              if (i < j) first = false;
              w += g.wts[t * g.k + i];
            }
        }
      }
      if (first) {
        row = rowof[e] + __popcll(mask[e] & ((1ull << t) - 1));
        wrow[row] = w;
      }
      srow[a] = row;
    }
  }
  c1.total = (int64_t)c1.ng * c1.mt * c1.nk;
  c1.P = (int)max((int64_t)1, min((int64_t)gridDim.x, c1.total / g.least));
  c2.total = (int64_t)c2.ng * c2.mt * c2.nk;
  c2.P = (int)max((int64_t)1, min((int64_t)gridDim.x, c2.total / g.least));
  if (c1.total == 0) c1.P = c2.P = 0;       // no token has an expert: nothing to claim
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_u = tc::smem_u32(full), empty_u = tc::smem_u32(empty);
  const uint32_t sa_u = tc::smem_u32(sa), sb_u = tc::smem_u32(sb);
  const int shares = c1.P + (LAYER ? c2.P : 0);

  // The n-th claimed share, by every role but the claiming one: -1 at the end or
  // where a wait ran out.
  auto take = [&](uint32_t n) -> int {
    if (!tc::mbar_wait(&qfull[n % kFQueue], (n / kFQueue) & 1, abort)) return -1;
    const int s = *reinterpret_cast<volatile int*>(&queue[n % kFQueue]);
    return s;
  };

  if (warp == 0) {
    // ---------------- claims, and the weights' copies ----------------
    if (lane == 0) {
      const uint64_t policy = tc::policy_evict_first();
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        int s = LAYER ? atomicAdd(g.ticket, 1) : (n == 0 ? (int)blockIdx.x : shares);
        if (s >= shares) s = -1;
        if (!tc::mbar_wait(&qempty[n % kFQueue], ((n / kFQueue) & 1) ^ 1, abort)) { ok = false; break; }
        queue[n % kFQueue] = s;
        tc::mbar_arrive(&qfull[n % kFQueue]);
        if (s < 0) break;
        const bool second = LAYER && s >= c1.P;
        const Cut& c = second ? c2 : c1;
        if (second) s -= c1.P;
        const int K = second ? g.K2 : g.K1, rows = second ? kFM : g.rows1;
        const CUtensorMap* map = &maps.a[second];
        const int64_t end = c.begin(s + 1);
        for (int64_t at = c.begin(s); ok && at < end;) {
          Piece p;
          if (second) piece_at<true>(c, at, end, p);
          else piece_at<false>(c, at, end, p);
          at = p.t0 + p.k1;
          const int e = LAYER ? glist[p.gi] : 0, f0 = p.j * rows;
          for (int kb = p.k0; kb < p.k1; ++kb) {
            if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
            const int k = kb * kFK, halves = K - k > kFH ? 2 : 1;
            tc::bar_arrive_expect_tx(full_u + 8 * slot, halves * kFA);
            for (int h = 0; h < halves; ++h)
              tma_weights(sa_u + (2 * slot + h) * kFA, map, k + h * kFH, f0, 0, e, full_u + 8 * slot, policy);
            ++issued;
            if (++slot == g.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
      }
      if (!ok || *abort) {
        // wind-down: the copies of this thread still in flight. A slot's barrier
        // completes only when the other copying warp arrived too; where that one
        // stopped earlier the limit ends the wait
        volatile int never = 0;
        const uint32_t left = issued < (uint32_t)g.stages ? issued : (uint32_t)g.stages;
        for (uint32_t k = 0; k < left; ++k) {
          const uint32_t i = issued - 1 - k;
          tc::mbar_wait(&full[i % g.stages], (i / g.stages) & 1, &never, 100000000ll);
        }
      }
    }
  } else if (warp == 2) {
    // ---------------- the rows' copies ----------------
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true, ready = false;
      for (uint32_t n = 0; ok; ++n) {
        int s = take(n);
        if (s < 0) break;
        const bool second = LAYER && s >= c1.P;
        const Cut& c = second ? c2 : c1;
        if (second) s -= c1.P;
        if (second && !ready) {
          // every tile of the first product has written its rows
          const int want = c1.ng * c1.mt;
          const long long t0 = clock64();
          for (uint32_t it = 1; ld_acquire_gpu(g.done) < want; ++it) {
            if ((it & 15) == 0 && (*abort || clock64() - t0 > 4000000000ll)) {
              *abort = 1;
              ok = false;
              break;
            }
          }
          if (!ok) break;
          fence_proxy_async_global();
          ready = true;
        }
        const int K = second ? g.K2 : g.K1;
        const int64_t end = c.begin(s + 1);
        for (int64_t at = c.begin(s); ok && at < end;) {
          Piece p;
          if (second) piece_at<true>(c, at, end, p);
          else piece_at<false>(c, at, end, p);
          at = p.t0 + p.k1;
          int r0 = 0, wide = g.N;
          const CUtensorMap* map = &maps.x;
          if (second) {
            const int e = glist[p.gi], m = __popcll(mask[e]);
            wide = (m + 15) & ~15;
            map = &maps.y[wide / 16 - 1];
            r0 = rowof[e];
          }
          for (int kb = p.k0; kb < p.k1; ++kb) {
            if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
            const int k = kb * kFK, halves = K - k > kFH ? 2 : 1;
            tc::bar_arrive_expect_tx(full_u + 8 * slot, halves * wide * 128);
            for (int h = 0; h < halves; ++h)
              tc::tma_load_2d_at(sb_u + (2 * slot + h) * b_half, map, k + h * kFH, r0, full_u + 8 * slot);
            ++issued;
            if (++slot == g.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        tc::mbar_arrive(&qempty[n % kFQueue]);
      }
      if (!ok || *abort) {
        volatile int never = 0;
        const uint32_t left = issued < (uint32_t)g.stages ? issued : (uint32_t)g.stages;
        for (uint32_t k = 0; k < left; ++k) {
          const uint32_t i = issued - 1 - k;
          tc::mbar_wait(&full[i % g.stages], (i / g.stages) & 1, &never, 100000000ll);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    if (lane == 0) {
      const uint64_t ad0 = tc::smem_desc_sw128(sa_u), bd0 = tc::smem_desc_sw128(sb_u);
      const uint32_t hi = (uint32_t)(ad0 >> 32), a_step = kFA / 16, b_step = b_half / 16;
      int slot = 0;
      uint32_t phase = 0, tiles = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        int s = take(n);
        if (s < 0) break;
        const bool second = LAYER && s >= c1.P;
        const Cut& c = second ? c2 : c1;
        if (second) s -= c1.P;
        const int K = second ? g.K2 : g.K1;
        const int64_t end = c.begin(s + 1);
        for (int64_t at = c.begin(s); ok && at < end; ++tiles) {
          Piece p;
          if (second) piece_at<true>(c, at, end, p);
          else piece_at<false>(c, at, end, p);
          at = p.t0 + p.k1;
          const int d = tiles & 1;
          if (!tc::mbar_wait(&accempty[d], ((tiles >> 1) & 1) ^ 1, abort)) { ok = false; break; }
          tc::fence_after_sync();
          const int wide = second ? (__popcll(mask[glist[p.gi]]) + 15) & ~15 : g.N;
          const uint32_t idesc = tc::idesc_16bit(kFM, wide, g.dtype == MOE_DT_BF16, 0, 0), dt = tmem + d * ncol;
          for (int kb = p.k0; kb < p.k1; ++kb) {
            if (!tc::bar_wait(full_u + 8 * slot, phase, abort)) { ok = false; break; }
            tc::fence_after_sync();
            const uint32_t a0 = (uint32_t)ad0 + 2 * slot * a_step, b0 = (uint32_t)bd0 + 2 * slot * b_step;
            tc::mma_f16_x4<1>(dt, a0, hi, 2, b0, hi, 2, idesc, kb > p.k0);
            if (K - kb * kFK > kFH) tc::mma_f16_x4<1>(dt, a0 + a_step, hi, 2, b0 + b_step, hi, 2, idesc, 1u);
            tc::bar_commit(empty_u + 8 * slot);
            if (++slot == g.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          tc::mma_commit(&accfull[d]);
        }
        tc::mbar_arrive(&qempty[n % kFQueue]);
      }
      // every MMA of this thread has completed once `drain` fires
      tc::mma_commit(drain);
      volatile int never = 0;
      tc::mbar_wait(drain, 0, &never, 400000000ll);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int et = tid - 128, q = warp & 3;               // et: the tile's lane
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const bool gated = act_gated(g.act.act);
    uint32_t tiles = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      int s = take(n);
      if (!epi_all(s >= 0)) break;
      const bool second = LAYER && s >= c1.P;
      const Cut& c = second ? c2 : c1;
      if (second) s -= c1.P;
      const int64_t end = c.begin(s + 1);
      for (int64_t at = c.begin(s); at < end; ++tiles) {
        Piece p;
        if (second) piece_at<true>(c, at, end, p);
        else piece_at<false>(c, at, end, p);
        at = p.t0 + p.k1;
        const int d = tiles & 1;
        const bool got = tc::mbar_wait(&accfull[d], (tiles >> 1) & 1, abort);
        if (!epi_all(got)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t acc = lanes + d * ncol;
        auto release = [&] {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&accempty[d]);
        };
        const int e = LAYER ? glist[p.gi] : 0;
        const unsigned long long toks = LAYER ? mask[e] : 0ull;
        const int m = LAYER ? __popcll(toks) : g.R;
        const bool head = p.k0 == 0, whole = head && p.k1 == c.nk;
        if (!second) {
          // columns of the group's tokens, kFCols at a time, each as 128 lanes' fp32
          auto columns = [&](unsigned long long& rem, int i0, int nc, uint32_t (&v)[kFCols]) {
#pragma unroll
            for (int i = 0; i < kFCols; ++i)
              if (i < nc) tmem_ld1(acc + (LAYER ? next_bit(rem) : i0 + i), v[i]);
            tc::tmem_wait_ld();
          };
          bool mine = whole;
          int s0 = s, s1 = s;
          if (!whole) {
            s0 = c.share_of(p.t0);
            s1 = c.share_of(p.t0 + c.nk - 1);
            float* to = g.part + (int64_t)(2 * s + head) * g.N * kFM;
            unsigned long long rem = toks;
            for (int i0 = 0; i0 < m; i0 += kFCols) {
              uint32_t v[kFCols];
              const int nc = min(kFCols, m - i0);
              columns(rem, i0, nc, v);
#pragma unroll
              for (int i = 0; i < kFCols; ++i)
                if (i < nc) to[(i0 + i) * kFM + et] = __uint_as_float(v[i]);
            }
            release();
            __threadfence();
            epi_sync();
            if (et == 0) {
              const int old = atom_add_acq_rel_gpu(&g.split[s0], 1);
              tmp[1] = old == s1 - s0;
              if (old == s1 - s0) g.split[s0] = 0;      // for the next call
            }
            epi_sync();
            mine = *reinterpret_cast<volatile int*>(&tmp[1]);
            __threadfence();
          }
          if (mine) {
            unsigned long long rem = toks;
            for (int i0 = 0; i0 < m; i0 += kFCols) {
              const int nc = min(kFCols, m - i0);
              float f[kFCols];
              if (whole) {
                uint32_t v[kFCols];
                columns(rem, i0, nc, v);
#pragma unroll
                for (int i = 0; i < kFCols; ++i) f[i] = __uint_as_float(v[i]);
              } else {
#pragma unroll
                for (int i = 0; i < kFCols; ++i) f[i] = 0.f;
                for (int w = s0; w <= s1; ++w) {
                  const float* from = g.part + (int64_t)(2 * w + (w == s0)) * g.N * kFM;
#pragma unroll
                  for (int i = 0; i < kFCols; ++i)
                    if (i < nc) f[i] += __ldcg(from + (i0 + i) * kFM + et);
                }
              }
#pragma unroll
              for (int i = 0; i < kFCols; ++i)
                if (i < nc) stage[i * kFM + et] = f[i];
              if (whole && i0 + kFCols >= m) release();
              epi_sync();
              const int F = gated ? 64 : 128;             // features of the tile
              for (int o = et; o < nc * F; o += 128) {
                const int i = o / F, l = o % F, f1 = p.j * F + l;
                if (f1 >= g.F1) continue;
                float a = stage[i * kFM + l], u = gated ? stage[i * kFM + 64 + l] : 0.f;
                if constexpr (LAYER) {
                  if (g.b1) {
                    a += g.b1[(int64_t)e * 2 * g.F1 + f1];
                    u += g.b1[(int64_t)e * 2 * g.F1 + g.F1 + f1];
                  }
                  const int row = rowof[e] + i0 + i;
                  const float y = gated ? act_two(a, u, g.act) : act_one(a, g.act.act);
                  reinterpret_cast<uint16_t*>(g.y)[(int64_t)row * g.ldy + f1] = E::from(wrow[row] * y);
                } else {
                  const int r = i0 + i;
                  if (g.bias) {
                    if (g.wdtype == MOE_DT_F32) {
                      const float* b = reinterpret_cast<const float*>(g.bias);
                      a += b[f1];
                      if (gated) u += b[g.F1 + f1];
                    } else {
                      const uint16_t* b = reinterpret_cast<const uint16_t*>(g.bias);
                      a += E::to(b[f1]);
                      if (gated) u += E::to(b[g.F1 + f1]);
                    }
                  }
                  if (g.z) {
                    uint16_t* z = reinterpret_cast<uint16_t*>(g.z) + r * g.ldz;
                    z[f1] = E::from(a);
                    if (gated) z[g.F1 + f1] = E::from(u);
                  }
                  float y = gated ? act_two(a, u, g.act) : act_one(a, g.act.act);
                  if (g.res) y += E::to(reinterpret_cast<const uint16_t*>(g.res)[r * g.ldr + f1]);
                  reinterpret_cast<uint16_t*>(g.out)[r * g.ldo + f1] = E::from(y);
                }
              }
              epi_sync();
            }
            if constexpr (LAYER) {
              // the rows of this tile are in memory, for the tensor copies of any CTA
              __threadfence();
              fence_proxy_async_global();
              epi_sync();
              if (et == 0) atom_add_acq_rel_gpu(g.done, 1);
            }
          }
        } else if constexpr (LAYER) {
          const int h = p.j * kFM + et;
          float* to = head ? g.zrow + (int64_t)rowof[e] * g.ldz32 + h : g.part + (int64_t)s * g.N * kFM + et;
          const int64_t step = head ? g.ldz32 : kFM;
          for (int i0 = 0; i0 < m; i0 += kFCols) {
            uint32_t v[kFCols];
#pragma unroll
            for (int i = 0; i < kFCols; ++i)
              if (i0 + i < m) tmem_ld1(acc + i0 + i, v[i]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kFCols; ++i)
              if (i0 + i < m) to[(i0 + i) * step] = __uint_as_float(v[i]);
          }
          release();
          // the share's last piece of this feature tile: whoever finishes it joins
          // the tokens' rows
          if (at < end && at / c.nk / c.ng == p.j) continue;
          const int64_t j0 = (int64_t)p.j * c.ng * c.nk;
          const int n_shares = c.share_of(j0 + (int64_t)c.ng * c.nk - 1) - c.share_of(j0) + 1;
          __threadfence();
          epi_sync();
          if (et == 0) {
            const int old = atom_add_acq_rel_gpu(&g.split2[p.j], 1);
            tmp[1] = old == n_shares - 1;
          }
          epi_sync();
          if (*reinterpret_cast<volatile int*>(&tmp[1])) {
            __threadfence();
            for (int t = 0; t < g.R; ++t) {
              float sum = 0.f;
              for (int j = 0; j < kp; ++j) {
                const int row = srow[t * kp + j];
                if (row < 0) continue;
                sum += __ldcg(g.zrow + (int64_t)row * g.ldz32 + h);
                // pieces of that group's tile in later shares
                const int eg = j < g.k ? g.ids[t * g.k + j] : g.E + j - g.k;
                int gi = 0;
                for (int lo = 0, hi = c.ng - 1; lo <= hi;) {
                  const int mid = (lo + hi) >> 1;
                  if (glist[mid] <= eg) { gi = mid; lo = mid + 1; } else hi = mid - 1;
                }
                const int64_t t0 = j0 + (int64_t)gi * c.nk;
                const int w1 = c.share_of(t0 + c.nk - 1);
                for (int w = c.share_of(t0) + 1; w <= w1; ++w)
                  sum += __ldcg(g.part + ((int64_t)w * g.N + row - rowof[eg]) * kFM + et);
              }
              if (h < g.F2) reinterpret_cast<uint16_t*>(g.out)[t * g.ldo + h] = E::from(sum);
            }
          }
        }
      }
      __syncwarp();
      if (warp == 4 && lane == 0) tc::mbar_arrive(&qempty[n % kFQueue]);
    }
  }

  if (LAYER && shares == 0 && blockIdx.x == 0)      // no token has an expert
    for (int64_t i = tid; i < (int64_t)g.R * g.F2; i += kFThreads)
      reinterpret_cast<uint16_t*>(g.out)[i / g.F2 * g.ldo + i % g.F2] = 0;
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort) set_status(g.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 2 * ncol);
  }
}

// ---- host -------------------------------------------------------------------------
static int64_t up(int64_t n, int64_t t) { return (n + t - 1) / t; }

// Weights [G][halves][rows][K]: boxes of 64 x 128 rows, gated 64 x 64 x both halves.
static bool map_weights(CUtensorMap* map, const void* w, int64_t K, int64_t rows, int halves, int64_t ld, int64_t G,
                        int64_t group) {
  const int64_t dims[4] = {K, rows, halves, G};
  const int64_t strides[3] = {ld, halves > 1 ? rows * ld : ld, G > 1 ? group : ld};
  const int box[4] = {kFH, kFM / halves, halves, 1};
  return make_tmap(map, w, 2, 4, dims, strides, box);
}
static bool map_rows(CUtensorMap* map, const void* x, int64_t K, int64_t rows, int64_t ld, int box_rows) {
  const int64_t dims[2] = {K, rows}, strides[1] = {ld};
  const int box[2] = {kFH, box_rows};
  return make_tmap(map, x, 2, 2, dims, strides, box);
}

template <typename E, bool LAYER>
static cudaError_t launch(FewArgs& g, const FewMaps& maps, cudaStream_t st) {
  const int G = g.E + g.S, kp = g.k + g.S;
  int head = kFBars + kFCols * kFM * 4;
  if (LAYER) head += 12 * G + 4 * std::min(G, g.R * kp) + 8 * g.R * kp + 64;
  g.head = (head + 1023) / 1024 * 1024;
  const int stage = 2 * (kFA + g.N * 128);
  g.stages = std::min(kFMaxStages, (kFSmem - 1024 - g.head) / stage);
  const int smem = 1024 + g.head + g.stages * stage;
  static std::atomic<bool> done[kMaxDevices] = {};
  const cudaError_t e = set_smem_once((const void*)k_few16<E, LAYER>, kFSmem, done);
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(k_few16<E, LAYER>, dim3(std::min(device_sms(), kFewShares)), dim3(kFThreads), smem, st, g, maps);
}

cudaError_t launch_few_layer(FewArgs g, const void* x, int64_t ldx, const void* w1, int64_t g1, int64_t ld1, const void* w2,
                             int64_t g2, int64_t ld2, cudaStream_t st) {
  const int G = g.E + g.S, halves = act_gated(g.act.act) ? 2 : 1;
  g.N = (g.R + 15) & ~15;
  g.rows1 = kFM / halves;
  g.mt1 = (int)up(g.F1, g.rows1); g.nk1 = (int)up(g.K1, kFK);
  g.mt2 = (int)up(g.F2, kFM); g.nk2 = (int)up(g.K2, kFK);
  g.least = 4;
  FewMaps maps;
  if (!map_weights(&maps.a[0], w1, g.K1, g.F1, halves, ld1, G, g1) || !map_weights(&maps.a[1], w2, g.K2, g.F2, 1, ld2, G, g2) ||
      !map_rows(&maps.x, x, g.K1, g.R, ldx, g.N))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 4; ++i)
    if (!map_rows(&maps.y[i], g.y, g.K2, (int64_t)g.R * (g.k + g.S), g.ldy, 16 * (i + 1))) return cudaErrorInvalidValue;
  return g.dtype == MOE_DT_BF16 ? launch<Bf16, true>(g, maps, st) : launch<F16, true>(g, maps, st);
}

cudaError_t launch_few_linear(FewArgs g, const void* x, int64_t ldx, const void* w, int64_t ldw, cudaStream_t st) {
  const int halves = act_gated(g.act.act) ? 2 : 1;
  g.N = (g.R + 15) & ~15;
  g.rows1 = kFM / halves;
  g.mt1 = (int)up(g.F1, g.rows1); g.nk1 = (int)up(g.K1, kFK);
  g.mt2 = g.nk2 = 0;
  g.least = 4;
  FewMaps maps = {};
  if (!map_weights(&maps.a[0], w, g.K1, g.F1, halves, ldw, 1, 0) || !map_rows(&maps.x, x, g.K1, g.R, ldx, g.N))
    return cudaErrorInvalidValue;
  return g.dtype == MOE_DT_BF16 ? launch<Bf16, false>(g, maps, st) : launch<F16, false>(g, maps, st);
}

}  // namespace moe
