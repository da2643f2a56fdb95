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
// A stage of weights: features f0 .. of group e (both halves of a gated tile),
// 64 of the reduction after 64. Where the reduction is a whole number of those
// the map has an axis of them and one copy brings the stage (a copy costs its
// thread some hundred cycles); else there is one for each 64 that exist.
__device__ __forceinline__ void copy_weights(uint32_t dst, int half_bytes, const CUtensorMap* map, bool chunks, int k, int n,
                                             int f0, int e, uint32_t bar, uint64_t policy) {
  for (int h = 0; h < (chunks ? 1 : n); ++h)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst + h * half_bytes),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(chunks ? 0 : k + h * kFH), "r"(f0), "r"(0), "r"(chunks ? k / kFH : 0), "r"(e),
        "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void copy_rows(uint32_t dst, int half_bytes, const CUtensorMap* map, bool chunks, int k, int n, int r0,
                                          uint32_t bar) {
  for (int h = 0; h < (chunks ? 1 : n); ++h)
    tc::tma_load_3d_at(dst + h * half_bytes, map, chunks ? 0 : k + h * kFH, r0, chunks ? k / kFH : 0, bar);
}
// Waits (bounded, whatever the abort flag says) for the copies that a thread still
// has in flight. A slot's barrier completes only when the other copying warp
// arrived too; where that one stopped earlier the limit ends the wait.
__device__ __forceinline__ void wind_down(uint64_t* full, uint32_t issued, int stages) {
  volatile int never = 0;
  const uint32_t left = issued < (uint32_t)stages ? issued : (uint32_t)stages;
  for (uint32_t k = 0; k < left; ++k) {
    const uint32_t i = issued - 1 - k;
    tc::mbar_wait(&full[i % stages], (i / stages) & 1, &never, 100000000ll);
  }
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

// out[t][128 j ..] = the rows of the token's slots, in slot order; a row's own
// pieces (a tile that spans shares) in order too. A warp a token, a lane four
// columns; the rows of four slots are asked for at once.
template <typename E>
__device__ __forceinline__ void join_tokens(const FewArgs& g, const Cut& c, int j, const int2* slot_of, int kp, int q, int lane) {
  const int h = j * kFM + 4 * lane;
  const int64_t j0 = (int64_t)j * c.ng * c.nk;
  const float* z = g.zrow + h;
  const bool vec = ((uintptr_t)g.out & 7) == 0 && g.ldo % 4 == 0 && h + 4 <= g.F2;
  for (int t = q; t < g.R; t += 4) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float4 v) { sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w; };
    for (int s = 0; s < kp; s += 8) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = s + i < kp ? slot_of[t * kp + s + i].x : -1;
        v[i] = row < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(reinterpret_cast<const float4*>(z + (int64_t)row * g.ldz32));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (s + i >= kp) break;
        const int2 sl = slot_of[t * kp + s + i];
        if (sl.x < 0) continue;
        add(v[i]);
        const int64_t t0 = j0 + (int64_t)(sl.y & 0xffff) * c.nk;
        const int w1 = c.share_of(t0 + c.nk - 1);
        for (int w = c.share_of(t0) + 1; w <= w1; ++w)
          add(__ldcg(reinterpret_cast<const float4*>(g.part + ((int64_t)w * g.N + (sl.y >> 16)) * kFM) + lane));
      }
    }
    uint16_t* o = reinterpret_cast<uint16_t*>(g.out) + t * g.ldo + h;
    if (vec) {
      *reinterpret_cast<uint2*>(o) = make_uint2(E::from2(sum.x, sum.y), E::from2(sum.z, sum.w));
    } else {
      if (h < g.F2) o[0] = E::from(sum.x);
      if (h + 1 < g.F2) o[1] = E::from(sum.y);
      if (h + 2 < g.F2) o[2] = E::from(sum.z);
      if (h + 3 < g.F2) o[3] = E::from(sum.w);
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kFThreads, 1) k_few_layer(const FewArgs g, const __grid_constant__ FewMaps maps) {
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
  int* rowof = reinterpret_cast<int*>(mask + G);        // [G] first row of the group
  int* glist = rowof + G;                               // [ng] groups with tokens
  int2* slot_of = reinterpret_cast<int2*>((reinterpret_cast<uintptr_t>(glist + min(G, g.R * kp)) + 7) & ~(uintptr_t)7);
  // slot_of [T kp]: row of a token's slot (-1: none); its group's place in glist and, from bit 16 on, its row in the group
  float* wrow = reinterpret_cast<float*>(slot_of + g.R * kp);   // [rows] routing weight
  int* gplace = reinterpret_cast<int*>(wrow + g.R * kp);        // [G] the group's place in glist
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
  for (int i = tid; i < G; i += kFThreads) mask[i] = i >= g.E ? (g.R == 64 ? ~0ull : (1ull << g.R) - 1) : 0ull;
  pdl_enter();
  __syncthreads();

  Cut c1 = {g.mt1, g.nk1, 1, 1, 0}, c2 = {g.mt2, g.nk2, 0, 1, 0};
  {
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
      gplace[e] = il;
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
      slot_of[a] = make_int2(row, first ? gplace[e] | (row - rowof[e]) << 16 : 0);
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
  const int shares = c1.P + c2.P;

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
        int s = atomicAdd(g.ticket, 1);
        if (s >= shares) s = -1;
        if (!tc::mbar_wait(&qempty[n % kFQueue], ((n / kFQueue) & 1) ^ 1, abort)) { ok = false; break; }
        queue[n % kFQueue] = s;
        tc::mbar_arrive(&qfull[n % kFQueue]);
        if (s < 0) break;
        const bool second = s >= c1.P;
        const Cut& c = second ? c2 : c1;
        if (second) s -= c1.P;
        const int K = second ? g.K2 : g.K1, rows = second ? kFM : g.rows1;
        const CUtensorMap* map = &maps.a[second];
        const bool chunks = K % kFH == 0;
        const int64_t end = c.begin(s + 1);
        for (int64_t at = c.begin(s); ok && at < end;) {
          Piece p;
          if (second) piece_at<true>(c, at, end, p);
          else piece_at<false>(c, at, end, p);
          at = p.t0 + p.k1;
          const int e = glist[p.gi], f0 = p.j * rows;
          for (int kb = p.k0; kb < p.k1; ++kb) {
            if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
            const int k = kb * kFK, n = chunks || K - k > kFH ? 2 : 1;
            tc::bar_arrive_expect_tx(full_u + 8 * slot, n * kFA);
            copy_weights(sa_u + 2 * slot * kFA, kFA, map, chunks, k, n, f0, e, full_u + 8 * slot, policy);
            ++issued;
            if (++slot == g.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
      }
      if (!ok || *abort) {
        wind_down(full, issued, g.stages);
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
        const bool second = s >= c1.P;
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
        const bool chunks = K % kFH == 0;
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
            const int k = kb * kFK, n = chunks || K - k > kFH ? 2 : 1;
            tc::bar_arrive_expect_tx(full_u + 8 * slot, n * wide * 128);
            copy_rows(sb_u + 2 * slot * b_half, wide * 128, map, chunks, k, n, r0, full_u + 8 * slot);
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
        wind_down(full, issued, g.stages);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    if (lane == 0) {
      const uint64_t ad0 = tc::smem_desc_sw128(sa_u), bd0 = tc::smem_desc_sw128(sb_u);
      const uint32_t hi = (uint32_t)(ad0 >> 32), a_step = kFA / 16;
      int slot = 0;
      uint32_t phase = 0, tiles = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        int s = take(n);
        if (s < 0) break;
        const bool second = s >= c1.P;
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
          const uint32_t idesc = tc::idesc_16bit(kFM, wide, g.dtype == MOE_DT_BF16, 0, 0), dt = tmem + d * ncol, b_step = wide * 8;
          for (int kb = p.k0; kb < p.k1; ++kb) {
            if (!tc::bar_wait(full_u + 8 * slot, phase, abort)) { ok = false; break; }
            tc::fence_after_sync();
            const uint32_t a0 = (uint32_t)ad0 + 2 * slot * a_step, b0 = (uint32_t)bd0 + slot * (b_half / 8);
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
      const bool second = s >= c1.P;
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
        const int e = glist[p.gi];
        const unsigned long long toks = mask[e];
        const int m = __popcll(toks);
        const bool head = p.k0 == 0, whole = head && p.k1 == c.nk;
        if (!second) {
          // columns of the group's tokens, kFCols at a time, each as 128 lanes' fp32
          auto columns = [&](unsigned long long& rem, int i0, int nc, uint32_t (&v)[kFCols]) {
#pragma unroll
            for (int i = 0; i < kFCols; ++i)
              if (i < nc) tmem_ld1(acc + (next_bit(rem)), v[i]);
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
                if (g.b1) {
                  a += g.b1[(int64_t)e * 2 * g.F1 + f1];
                  u += g.b1[(int64_t)e * 2 * g.F1 + g.F1 + f1];
                }
                const int row = rowof[e] + i0 + i;
                const float y = gated ? act_two(a, u, g.act) : act_one(a, g.act.act);
                reinterpret_cast<uint16_t*>(g.y)[(int64_t)row * g.ldy + f1] = E::from(wrow[row] * y);
              }
              epi_sync();
            }
            // the rows of this tile are in memory, for the tensor copies of any CTA
            __threadfence();
            fence_proxy_async_global();
            epi_sync();
            if (et == 0) atom_add_acq_rel_gpu(g.done, 1);
          }
        } else {
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
            join_tokens<E>(g, c, p.j, slot_of, kp, q, lane);
          }
        }
      }
      __syncwarp();
      if (warp == 4 && lane == 0) tc::mbar_arrive(&qempty[n % kFQueue]);
    }
  }

  if (shares == 0 && blockIdx.x == 0)      // no token has an expert
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

// ---- one dense product ------------------------------------------------------------
// Tiles of f features (a multiple of 8, gated: of each half) x N rows over the
// whole reduction, sized so that their rounds over the SMs come out even: with
// weights on the M side a tile of 48 features costs 48 rows of copies, and what
// the MMA computes for the other lanes is not read. (Cutting fixed tiles along
// the reduction instead costs the partial sums' way through memory: 1 x 7168 x
// 2048 13.9 us, 64 rows 86 us.)
constexpr int kLStages = 32;
constexpr int kLThreads = 384;
constexpr int kLChunk = 16;           // columns the epilogue takes at a time
constexpr int kLHead = 1024;          // barriers
constexpr int kLBias = 2 * kLChunk * kFM;     // gated: where a tile's biases lie in the epilogue's memory, two tiles'

template <typename E, bool GATED>
__global__ void __launch_bounds__(kLThreads, 1) k_few_linear(const FewArgs g, const __grid_constant__ FewMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* empty = full + kLStages;
  uint64_t* accfull = empty + kLStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* stage = reinterpret_cast<float*>(base + kLHead);           // gated: [2][kLChunk][128], biases [2][128]
  const int a_half = (GATED ? 2 : 1) * g.rows1 * 128, b_half = g.N * 128;
  uint8_t* sb = base + g.head;
  uint8_t* sa = sb + g.stages * 2 * b_half;                         // behind it 16 KB that MMAs may read
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) {
      tc::mbar_init(&full[i], 2);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], 1);
      tc::mbar_init(&accempty[i], 8);
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.a[0]);
    tc::prefetch_tmap(&maps.x);
  }
  const uint32_t ncol = g.N <= 32 ? 32 : g.N <= 64 ? 64 : g.N <= 128 ? 128 : 256;
  if (warp == 1) tc::tmem_alloc(tmem_slot, 2 * ncol);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_enter();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_u = tc::smem_u32(full), empty_u = tc::smem_u32(empty);
  const uint32_t sa_u = tc::smem_u32(sa), sb_u = tc::smem_u32(sb);
  const int tiles = g.mt1 * g.nt;
  const bool chunks = g.K1 % kFH == 0;

  if (warp == 0 || warp == 2) {
    // ---------------- copies: warp 0 weights, warp 2 rows ----------------
    if (lane == 0) {
      // weights that several row tiles read are worth keeping
      const uint64_t policy = g.nt > 1 ? tc::policy_evict_last() : tc::policy_evict_first();
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int f0 = t / g.nt * g.rows1, r0 = t % g.nt * g.N;
        for (int kb = 0; kb < g.nk1; ++kb) {
          if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
          const int k = kb * kFK, n = chunks || g.K1 - k > kFH ? 2 : 1;
          const uint32_t bar = full_u + 8 * slot;
          if (warp == 0) {
            tc::bar_arrive_expect_tx(bar, n * a_half);
            copy_weights(sa_u + 2 * slot * a_half, a_half, &maps.a[0], chunks, k, n, f0, 0, bar, policy);
          } else {
            tc::bar_arrive_expect_tx(bar, n * b_half);
            copy_rows(sb_u + 2 * slot * b_half, b_half, &maps.x, chunks, k, n, r0, bar);
          }
          ++issued;
          if (++slot == g.stages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok || *abort) wind_down(full, issued, g.stages);
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    if (lane == 0) {
      const uint64_t ad0 = tc::smem_desc_sw128(sa_u), bd0 = tc::smem_desc_sw128(sb_u);
      const uint32_t hi = (uint32_t)(ad0 >> 32), a_step = a_half / 16, b_step = b_half / 16;
      const uint32_t idesc = tc::idesc_16bit(kFM, g.N, g.dtype == MOE_DT_BF16, 0, 0);
      int slot = 0;
      uint32_t phase = 0, done = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++done) {
        const int d = done & 1;
        if (!tc::mbar_wait(&accempty[d], ((done >> 1) & 1) ^ 1, abort)) break;
        tc::fence_after_sync();
        const uint32_t dt = tmem + d * ncol;
        for (int kb = 0; kb < g.nk1; ++kb) {
          if (!tc::bar_wait(full_u + 8 * slot, phase, abort)) { ok = false; break; }
          tc::fence_after_sync();
          const uint32_t a0 = (uint32_t)ad0 + 2 * slot * a_step, b0 = (uint32_t)bd0 + 2 * slot * b_step;
          tc::mma_f16_x4<1>(dt, a0, hi, 2, b0, hi, 2, idesc, kb > 0);
          if (g.K1 - kb * kFK > kFH) tc::mma_f16_x4<1>(dt, a0 + a_step, hi, 2, b0 + b_step, hi, 2, idesc, 1u);
          tc::bar_commit(empty_u + 8 * slot);
          if (++slot == g.stages) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (ok) tc::mma_commit(&accfull[d]);
      }
      // every MMA of this thread has completed once `drain` fires
      tc::mma_commit(drain);
      volatile int never = 0;
      tc::mbar_wait(drain, 0, &never, 400000000ll);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    // Two groups of four warps share a tile's columns, kLChunk by kLChunk. A
    // lane holds a feature; the gate and up of a gated tile lie in different
    // lanes and meet in shared memory.
    const int grp = (warp - 4) >> 2, q = warp & 3, et = (threadIdx.x - 128) & 127;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    float* st = stage + grp * kLChunk * kFM;
    const uint16_t* res = reinterpret_cast<const uint16_t*>(g.res);
    uint16_t *z = reinterpret_cast<uint16_t*>(g.z), *out = reinterpret_cast<uint16_t*>(g.out);
    auto bias = [&](int64_t f) {
      return !g.bias ? 0.f : g.wdtype == MOE_DT_F32 ? reinterpret_cast<const float*>(g.bias)[f]
                                                   : E::to(reinterpret_cast<const uint16_t*>(g.bias)[f]);
    };
    auto group_sync = [&] {
      __syncwarp();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
    };
    uint32_t done = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++done) {
      const int d = done & 1, f0 = t / g.nt * g.rows1, r0 = t % g.nt * g.N, nr = min(g.N, g.R - r0);
      const int nf = min(g.rows1, g.F1 - f0);                       // features of the tile
      const uint32_t acc = lanes + d * ncol;
      float b0 = 0.f;
      if (et < nf) {
        b0 = bias(f0 + et);
        if (GATED && grp == 0) {
          stage[kLBias + d * kFM + et] = b0;
          stage[kLBias + d * kFM + 64 + et] = bias((int64_t)g.F1 + f0 + et);
        }
      }
      const bool got = tc::mbar_wait(&accfull[d], (done >> 1) & 1, abort);
      // what one of the eight warps gives up, all do: they meet at barriers below
      uint32_t all;
      __syncwarp();
      asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 3, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
                   : "=r"(all)
                   : "r"((uint32_t)got)
                   : "memory");
      if (!all) break;
      tc::fence_after_sync();
      for (int c = grp * kLChunk; c < nr; c += 2 * kLChunk) {
        const int n = min(kLChunk, nr - c);
        uint32_t v[kLChunk];
        tc::tmem_ld16(acc + c, v);
        tc::tmem_wait_ld();
        if constexpr (!GATED) {
          if (et < nf) {
            const int64_t f = f0 + et, r = r0 + c;
            float rv[kLChunk];
#pragma unroll
            for (int i = 0; i < kLChunk; ++i) rv[i] = res && i < n ? E::to(res[(r + i) * g.ldr + f]) : 0.f;
#pragma unroll
            for (int i = 0; i < kLChunk; ++i) {
              if (i >= n) break;
              const float a = __uint_as_float(v[i]) + b0;
              if (z) z[(r + i) * g.ldz + f] = E::from(a);
              out[(r + i) * g.ldo + f] = E::from(act_one(a, g.act.act) + rv[i]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kLChunk; ++i) st[i * kFM + et] = __uint_as_float(v[i]);
          group_sync();
          const float* bs = stage + kLBias + d * kFM;
          for (int o = et; o < n * 64; o += 128) {
            const int i = o >> 6, l = o & 63;
            if (l >= nf) continue;
            const int64_t f = f0 + l, r = r0 + c + i;
            const float a = st[i * kFM + l] + bs[l], u = st[i * kFM + g.rows1 + l] + bs[64 + l];
            if (z) {
              z[r * g.ldz + f] = E::from(a);
              z[r * g.ldz + g.F1 + f] = E::from(u);
            }
            const float y = act_two(a, u, g.act);
            out[r * g.ldo + f] = E::from(res ? y + E::to(res[r * g.ldr + f]) : y);
          }
          group_sync();
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&accempty[d]);
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) set_status(g.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 2 * ncol);
  }
}

// ---- host -------------------------------------------------------------------------
static int64_t up(int64_t n, int64_t t) { return (n + t - 1) / t; }

// Weights [G][halves][rows][K]: boxes of 64 x box rows x halves, twice along K
// where K is a whole number of 64 (see copy_weights).
static bool map_weights(CUtensorMap* map, const void* w, int64_t K, int64_t rows, int halves, int64_t ld, int64_t G,
                        int64_t group, int box_rows) {
  const bool chunks = K % kFH == 0;
  const int64_t dims[5] = {chunks ? kFH : K, rows, halves, chunks ? K / kFH : 1, G};
  const int64_t strides[4] = {ld, halves > 1 ? rows * ld : ld, chunks ? kFH : ld, G > 1 ? group : ld};
  const int box[5] = {kFH, box_rows, halves, chunks ? 2 : 1, 1};
  return make_tmap(map, w, 2, 5, dims, strides, box);
}
static bool map_rows(CUtensorMap* map, const void* x, int64_t K, int64_t rows, int64_t ld, int box_rows) {
  const bool chunks = K % kFH == 0;
  const int64_t dims[3] = {chunks ? kFH : K, rows, chunks ? K / kFH : 1}, strides[2] = {ld, chunks ? kFH : ld};
  const int box[3] = {kFH, box_rows, chunks ? 2 : 1};
  return make_tmap(map, x, 2, 3, dims, strides, box);
}

template <typename E>
static cudaError_t launch_layer(FewArgs& g, const FewMaps& maps, cudaStream_t st) {
  const int G = g.E + g.S, kp = g.k + g.S;
  const int head = kFBars + kFCols * kFM * 4 + 16 * G + 4 * std::min(G, g.R * kp) + 12 * g.R * kp + 64;
  g.head = (head + 1023) / 1024 * 1024;
  const int stage = 2 * (kFA + g.N * 128);
  g.stages = std::min(kFMaxStages, (kFSmem - 1024 - g.head) / stage);
  const int smem = 1024 + g.head + g.stages * stage;
  static std::atomic<bool> done[kMaxDevices] = {};
  const cudaError_t e = set_smem_once((const void*)k_few_layer<E>, kFSmem, done);
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(k_few_layer<E>, dim3(std::min(device_sms(), kFewShares)), dim3(kFThreads), smem, st, g, maps);
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
  if (!map_weights(&maps.a[0], w1, g.K1, g.F1, halves, ld1, G, g1, g.rows1) ||
      !map_weights(&maps.a[1], w2, g.K2, g.F2, 1, ld2, G, g2, kFM) || !map_rows(&maps.x, x, g.K1, g.R, ldx, g.N))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 4; ++i)
    if (!map_rows(&maps.y[i], g.y, g.K2, (int64_t)g.R * (g.k + g.S), g.ldy, 16 * (i + 1))) return cudaErrorInvalidValue;
  return g.dtype == MOE_DT_BF16 ? launch_layer<Bf16>(g, maps, st) : launch_layer<F16>(g, maps, st);
}

template <typename E, bool GATED>
static cudaError_t launch_linear(FewArgs& g, const FewMaps& maps, int grid, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices] = {};
  const cudaError_t e = set_smem_once((const void*)k_few_linear<E, GATED>, kFSmem, done);
  if (e != cudaSuccess) return e;
  const int stage = 2 * 128 * ((GATED ? 2 : 1) * g.rows1 + g.N);
  g.head = (kLHead + (GATED ? (kLBias + 2 * kFM) * 4 : 0) + 1023) / 1024 * 1024;
  g.stages = std::min(kLStages, (kFSmem - 1024 - g.head - kFA) / stage);
  note_launch();
  return launch_pdl(k_few_linear<E, GATED>, dim3(grid), dim3(kLThreads), 1024 + g.head + g.stages * stage + kFA, st, g, maps);
}

cudaError_t launch_few_linear(FewArgs g, const void* x, int64_t ldx, const void* w, int64_t ldw, cudaStream_t st) {
  const bool gated = act_gated(g.act.act);
  const int halves = gated ? 2 : 1, sms = device_sms();
  // the tile with the least to copy: rounds over the SMs times its rows of both
  // operands, and a fixed cost of a round
  int64_t least = INT64_MAX;
  for (int nt = (int)up(g.R, 256); nt <= up(g.R, 16); ++nt) {
    const int n = (int)(up(up(g.R, nt), 16) * 16);
    if (up(g.R, n) != nt) continue;
    for (int f = kFM / halves; f >= 8; f -= 8) {
      if (f * halves + n > 256) continue;       // three stages at least
      const int64_t cost = up(up(g.F1, f) * nt, sms) * (f * halves + n + 16);
      if (cost < least) {
        least = cost;
        g.rows1 = f; g.N = n; g.nt = nt;
      }
    }
  }
  g.mt1 = (int)up(g.F1, g.rows1); g.nk1 = (int)up(g.K1, kFK);
  FewMaps maps = {};
  if (!map_weights(&maps.a[0], w, g.K1, g.F1, halves, ldw, 1, 0, g.rows1) || !map_rows(&maps.x, x, g.K1, g.R, ldx, g.N))
    return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>((int64_t)g.mt1 * g.nt, sms);
  if (gated)
    return g.dtype == MOE_DT_BF16 ? launch_linear<Bf16, true>(g, maps, grid, st) : launch_linear<F16, true>(g, maps, grid, st);
  return g.dtype == MOE_DT_BF16 ? launch_linear<Bf16, false>(g, maps, grid, st) : launch_linear<F16, false>(g, maps, grid, st);
}

}  // namespace moe
