// Products of 16-bit weights with a few rows, on the 5th-generation tensor cores,
// in one launch: the routed layer's both products with the activation and the
// combine, or one dense product with its epilogue.
//
// Bound: the weights' bytes; at small sizes latency. Everything else is arranged
// around the weights' stream.
//
// - Weights are the MMA's M side, the rows its N (16 to 256). The layer's first
//   product multiplies every expert's weights with all the tokens: up to 64
//   columns cost the tensor core little more than 16, and no gather is needed. The
//   epilogue reads the columns of the expert's own tokens; what the others hold
//   never leaves tensor memory, so a NaN stays with its token.
// - Each CTA takes an equal range of features over the whole reduction, wherever
//   it begins: of the first product a range of all touched experts' features, of
//   the second one of H, for which it runs through all touched experts (or, where
//   the range would be narrow, half or a quarter of them) and adds their columns to
//   the tokens' fp32 sums in shared memory. So no reduction is cut
//   (with tiles of 128 features cut along the reduction into equal shares, whose
//   partial sums the last CTA added, one token through 7168 x 2048 x 8 experts
//   took 127 us behind the router, 2880 x 2880 x 4 51, 256 x 128 x 2 20). A
//   tile's copies may cover a few rows of its neighbour, which the L2 serves.
// - The second product's weights do not depend on the first one: their copies run
//   ahead into the ring while the CTA's copies of the rows wait for all of the
//   first product, so the barrier between them costs no stream time as long as it
//   is shorter than the ring.
// - CTAs claim their ranges from a counter, all of the first product's before any
//   of the second's: a CTA that waits only waits for ranges that running CTAs
//   hold, however many of the grid are resident.
//
// Roles: warp 0 claims and copies weights, warp 2 copies rows, warps 1 and 3 and the
// last two issue the MMAs, those between are the epilogue (two accumulators, so that it
// overlaps the next tile's MMAs). An MMA takes its issuer some 60 cycles, however few
// its rows, and each stage a wait, a commit and the latency between them: with one
// issuer a half stage of 24 rows took 350 cycles, of which its copies need 130. So four
// warps issue, into an accumulator of their own each, and the epilogue adds the four.
// In the layer each takes one step (K = 16) in four of every stage, which is done
// the sooner (of a group of more than 32 tokens, whose two parts of y take 128 columns, two
// of them take two each); a dense product, whose calls are shorter, is the faster with whole
// stages in turn (16 x 2 x 2048 x 7168 13.5 us against 18.0; the layer 16 tokens, 2880 x 2880
// 394 against 379). Every wait is bounded; a CTA whose wait runs out sets
// MOE_DEV_TIMEOUT, waits for its copies and MMAs in flight, frees tensor memory and
// returns.
//
// Measured, in us, with ready ids (bf16, SwiGLU; in brackets the bytes that the
// tokens' experts need, at 6775 GB/s): 1 token x 7168 x 2048, 8 of 256 experts 114
// (105); 8 tokens 742 (748 for that many at random); 16 tokens x
// 2880 x 2880, 4 of 128, 370 (375); x 4096 x 512, 8 of 256, 203 (190); 64 tokens x 7168 x 2048, 8 of
// 64, 868 (832); x 2048 x 768, 8 of 128, 198 (176); 1 token x 2880 x 2880, 4 of 128, 45 (29); 1 token x
// 256 x 128, 2 of 8, 13.0 (latency); GPUs of one kind differ by 3 %, this is one of the slower. With
// 16 tokens and 24 experts the memory reads 1.015 times the weights' bytes, at 75 %
// of its time, the tensor pipe is 7 % busy.
#include <cmath>
#include <type_traits>

#include "few16.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kFM = 128;              // most features a tile (MMA M)
constexpr int kFH = 64;               // reduction of a half stage: one 128-byte swizzle row
constexpr int kFThreads = 320;
constexpr int kFMaxStages = 8;
constexpr int kFBars = 512;           // barriers and scratch, in front of the tables
constexpr int kFSmem = 227 * 1024;
constexpr int kFCols = 8;             // columns the layer's epilogue takes at a time (16 where there are no more)
constexpr int kFQueue = 4;            // claimed ranges in flight
constexpr int kFIssuers = 4;          // warps that issue the layer's MMAs
constexpr int kFLeast = 8;            // features a range, at least
constexpr int kFWide = 128;           // columns of an accumulator of the second product with more than 32 tokens

struct FewMaps {
  CUtensorMap a[8];                   // weights of the (first) product: boxes of 8 (i + 1) features (not gated: 16 (i + 1)),
                                      // dense: a[0], the tile's
  CUtensorMap a2;                     // layer: of the second
  CUtensorMap x;                      // rows of the (first) product
  CUtensorMap y[4];                   // layer: rows of the second, boxes of 8 << i, of each part
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr) : "memory");
}
// A stage of weights: features f0 .. of group e (both halves of a gated tile), n
// times 64 of the reduction. Where the reduction is a whole number of those the map
// has an axis of them and a copy brings two (a copy costs its thread some hundred
// cycles); else there is one for each 64.
__device__ __forceinline__ void copy_weights(uint32_t dst, int half_bytes, const CUtensorMap* map, bool chunks, int k, int n,
                                             int f0, int e, uint32_t bar, uint64_t policy) {
  for (int h = 0; h < n; h += chunks ? 2 : 1)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst + h * half_bytes),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(chunks ? 0 : k + h * kFH), "r"(f0), "r"(0), "r"(chunks ? k / kFH + h : 0), "r"(e),
        "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void copy_rows(uint32_t dst, int half_bytes, const CUtensorMap* map, bool chunks, int k, int n, int r0,
                                          uint32_t bar) {
  for (int h = 0; h < n; h += chunks ? 2 : 1)
    tc::tma_load_3d_at(dst + h * half_bytes, map, chunks ? 0 : k + h * kFH, r0, chunks ? k / kFH + h : 0, bar);
}
// Rows of the layer's second product, of both parts.
__device__ __forceinline__ void copy_y(uint32_t dst, int half_bytes, const CUtensorMap* map, bool chunks, int k, int n, int r0,
                                       uint32_t bar) {
  for (int h = 0; h < n; h += chunks ? 2 : 1)
    tc::tma_load_4d_at(dst + h * half_bytes, map, chunks ? 0 : k + h * kFH, r0, 0, chunks ? k / kFH + h : 0, bar);
}
// Where the way along the reduction, of ns stages, begins for range (tile) s: a small part of the way further for
// each, not at the same columns for all, whose rows lie a fixed distance apart. Not by CTA: which one takes a range
// varies, and sums must not. It is worth little, and not always that. In us, from the first column on, an
// eleventh further, and the golden ratio's part: dense 1 x 4096 x 4096 9.9, 9.5, 9.9; 16 x 2 x 2048 x 7168 13.4, 13.5, 13.8; 4 x
// 4096 x 14336 22.5, 22.7, 23.4; layer, 1 token x 7168 x 2048 122.6, 122.0, 122.0; x 4096 x 512 38.2, 38.7, 39.9; 16 x 2880 x 2880
// 379, 381, 381; 64 tokens 794, 796, 795.
__device__ __forceinline__ int first_stage(int s, int ns) {
  return (int)(((uint32_t)s * 5851u & 0xffffu) * (uint32_t)ns >> 16);      // an eleventh
}
// Most 64s of a reduction of K that a stage should hold (an even number): an eighth,
// so that a short reduction is shared among the issuers too.
__host__ __device__ __forceinline__ int stage_halves(int K) { return 2 * (1 + K / (16 * kFH)); }
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
__device__ __forceinline__ float add4(const uint32_t (&v)[4]) {
  return (__uint_as_float(v[0]) + __uint_as_float(v[1])) + (__uint_as_float(v[2]) + __uint_as_float(v[3]));
}
// C columns of the J accumulators (two or four), `apart` columns apart, added.
template <int C, int J = 4>
__device__ __forceinline__ void add_columns(uint32_t (&v)[C], uint32_t acc, uint32_t apart) {
  uint32_t u[J][C];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if constexpr (C == 16) tc::tmem_ld16(acc + j * apart, u[j]);
    else tmem_ld8(acc + j * apart, u[j]);
  }
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (J == 4) {
      const uint32_t w[4] = {u[0][i], u[1][i], u[2][i], u[3][i]};
      v[i] = __float_as_uint(add4(w));
    } else {
      v[i] = __float_as_uint(__uint_as_float(u[0][i]) + __uint_as_float(u[1][i]));
    }
  }
}
// What the first part of y is a multiple of. An f16 number ends at 65504, which squared ReLU passes at 256; in
// steps of 4096 the first part reaches 2^28, and what its rounding leaves, at most 2^-11 of it or 2^-13, the
// second holds to the 2^-25 that it would be off by in any case.
template <typename E>
__device__ constexpr float y_unit() {
  return std::is_same_v<E, F16> ? 4096.f : 1.f;
}
// The layer's epilogue warps only.
__device__ __forceinline__ void epi_sync() { __syncwarp(); asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Whether `ok` holds for all threads of `count` (barrier id): what one of them
// gives up, all do.
template <int ID, int COUNT>
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(ID), "n"(COUNT)
      : "memory");
  return r != 0;
}

// An MMA, four (the steps of 64 of the reduction) and a commit (see tc::bar_commit) by
// one thread of a warp that runs as a whole: the compiler then keeps addresses and
// descriptors in uniform registers, where the instructions want them (a thread of its
// own takes 67 cycles for an MMA, this 52 to 64, and its loop's own work on top of that).
__device__ __forceinline__ void mma_one(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_four(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n elect.sync _|q, 0xffffffff;\n"
      " setp.ne.b32 p, %11, 0;\n setp.eq.u32 t, 0, 0;\n"
      " mov.b64 a0, {%1, %9};\n mov.b64 b0, {%5, %9};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %10, p;\n"
      " mov.b64 a1, {%2, %9};\n mov.b64 b1, {%6, %9};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %10, t;\n"
      " mov.b64 a2, {%3, %9};\n mov.b64 b2, {%7, %9};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %10, t;\n"
      " mov.b64 a3, {%4, %9};\n mov.b64 b3, {%8, %9};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %10, t;\n}" ::"r"(d),
      "r"(a), "r"(a + 2), "r"(a + 4), "r"(a + 6), "r"(b), "r"(b + 2), "r"(b + 4), "r"(b + 6), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}
// A value that all lanes hold, in a uniform register.
__device__ __forceinline__ uint32_t uni(uint32_t v) { return __shfl_sync(kFull, v, 0); }

// Position of the lowest set bit, which is cleared.
__device__ __forceinline__ int next_bit(unsigned long long& m) {
  const int b = __ffsll((long long)m) - 1;
  m &= m - 1;
  return b;
}
// Copies cover 8 << i rows, the fewest that hold n.
__device__ __forceinline__ int box_of(int n) { return n <= 8 ? 0 : n <= 16 ? 1 : n <= 32 ? 2 : 3; }

// ---- the routed layer ---------------------------------------------------------------
// A tile: `len` features from f0 of group e, copied in boxes of `box` (gated: of
// each half): arows rows of the MMA's operand A. rows: of B that are copied; N: the
// MMA's. hs: 64s of the reduction a stage, an even number; ns: stages. Every role finds
// its tiles by itself, so no division is among the steps to the next one.
struct FewTile {
  int e, f0, len, bi, box, arows, rows, N, hs, ns;
};
// Runs through the tiles of a range, of `left` features from f0 of the g-th group. First
// product: over all groups' features one after the other, up to 64 (gated) or 128 a tile. Second: over
// features of H, up to 128 (the map's box) a tile, for each all groups [g0, g1), or one of g.S2 parts of them.
struct FewRange {
  int f0, left, g, g0, g1;
};
// a / b of a < 2^39 or so, mostly of 32 bits.
__device__ __forceinline__ int64_t div_short(int64_t a, int b) {
  return a < (1ll << 32) ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
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
  int* queue = reinterpret_cast<int*>(drain + kFIssuers);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(queue + kFQueue);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tmp = reinterpret_cast<int*>(tmem_slot + 2);                 // 1 + 2 * 10
  // the epilogue's answer to whether a part of a range was the last to be done. A word of its own: a warp without
  // a tile may read tmp[0], the groups, after the epilogue's first range
  volatile int* last = tmp + 21;
  float* stage = reinterpret_cast<float*>(base + kFBars);           // [16][128]
  const int G = g.E + g.S, A = g.R * g.k;
  const bool gated = act_gated(g.act.act);
  // the tokens' sums [T][g.box2]; then the tables
  float* sums = stage + 16 * kFM;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(sums + ((g.R * g.box2 + 1) & ~1));   // [G] tokens
  int* rowof = reinterpret_cast<int*>(mask + G);                    // [G] first row of the group
  int* glist = rowof + G;                                           // groups with tokens
  float* wrow = reinterpret_cast<float*>(glist + min(G, A + g.S));  // [rows] routing weight
  int* sid = reinterpret_cast<int*>(wrow + A + g.S * g.R);          // [A] the ids, -1: left out
  float* swt = reinterpret_cast<float*>(sid + A);                   // [A] their weights
  uint8_t* tokof = reinterpret_cast<uint8_t*>(swt + A);             // [rows] token
  uint8_t* ring = base + g.head;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < g.stages; ++i) {
      tc::mbar_init(&full[i], 2);
      tc::mbar_init(&empty[i], kFIssuers);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], kFIssuers);
      tc::mbar_init(&accempty[i], 4);
    }
    for (int i = 0; i < kFQueue; ++i) {
      tc::mbar_init(&qfull[i], 1);
      tc::mbar_init(&qempty[i], 2 + kFIssuers);     // rows' copies, epilogue, MMAs
    }
    for (int i = 0; i < kFIssuers; ++i) tc::mbar_init(&drain[i], 1);
    *abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 3 && lane < (int)(sizeof(FewMaps) / sizeof(CUtensorMap))) tc::prefetch_tmap(&maps.a[0] + lane);
  const uint32_t ncol = g.ncol;         // four accumulators a tile, two tiles
  if (warp == 1) tc::tmem_alloc(tmem_slot, 8 * ncol);
  for (int i = tid; i < G; i += kFThreads) mask[i] = i >= g.E ? (g.R == 64 ? ~0ull : (1ull << g.R) - 1) : 0ull;
  pdl_enter();
  // the first claim's answer passes behind the tables
  int claim = 0;
  if (tid == 0) claim = atomicAdd(g.ticket, 1);
  __syncthreads();

  // the tokens of every expert; an assignment of weight 0 is left out
  for (int a = tid; a < A; a += kFThreads) {
    int e = g.ids[a];
    const float w = g.wts[a];
    if (e < 0 || e >= g.E) {
      if (blockIdx.x == 0) set_status(g.status, MOE_DEV_BAD_EXPERT_ID);
      e = -1;
    } else if (w != 0.f) {
      atomicOr(&mask[e], 1ull << (a / g.k));
    }
    sid[a] = e;
    swt[a] = w;
  }
  __syncthreads();
  // groups with tokens, and every group's first row: prefix sums over the groups
  {
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
    if (lane == 31) { tmp[1 + warp] = il; tmp[11 + warp] = ir; }
    __syncthreads();
    il -= live;
    ir -= rows;
    for (int w = 0; w < warp; ++w) { il += tmp[1 + w]; ir += tmp[11 + w]; }
    for (int e = e0; e < e1; ++e) {
      rowof[e] = ir;
      if (mask[e]) glist[il++] = e;
      const int m = __popcll(mask[e]);
      if (e >= g.E)
        for (int i = 0; i < m; ++i) {
          wrow[ir + i] = 1.f;
          tokof[ir + i] = (uint8_t)i;
        }
      ir += m;
    }
    if (tid == kFThreads - 1) tmp[0] = il;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // a row's weight, by and for the epilogue's warps: a repeated id's weights add up, in slot order
  for (int a = tid - 128; warp >= 4 && warp < 8 && a < A; a += 128) {
    const int t = a / g.k, e = sid[a];
    if (e < 0 || !(mask[e] >> t & 1)) continue;
    bool first = true;
    float w = 0.f;
    for (int i = t * g.k; i < (t + 1) * g.k; ++i)
      if (sid[i] == e) {
        if (i < a) first = false;
        w += swt[i];
      }
    if (first) {
      const int r = rowof[e] + __popcll(mask[e] & ((1ull << t) - 1));
      wrow[r] = w;
      tokof[r] = (uint8_t)t;
    }
  }
  const int ng = tmp[0];
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_u = tc::smem_u32(full), empty_u = tc::smem_u32(empty), ring_u = tc::smem_u32(ring);
  const int64_t total1 = (int64_t)ng * g.F1;
  // ranges of both products; without a token that has an expert only the second's, of zeros
  const int P1 = (int)min((int64_t)gridDim.x, (total1 + kFLeast - 1) / kFLeast);
  const int P2 = g.Pf * g.S2;

  // The n-th claimed range, by every role but the claiming one: -1 at the end or
  // where a wait ran out.
  auto take = [&](uint32_t n) -> int {
    if (!tc::mbar_wait(&qfull[n % kFQueue], (n / kFQueue) & 1, abort)) return -1;
    return *reinterpret_cast<volatile int*>(&queue[n % kFQueue]);
  };
  auto range_of = [&](int s) -> FewRange {
    if (s < P1) {
      const int64_t at = div_short(total1 * s, P1), gi = div_short(at, g.F1);
      return {(int)(at - gi * g.F1), (int)(div_short(total1 * (s + 1), P1) - at), (int)gi, 0, 0};
    }
    // F2 <= 2^20, at most kFewSms ranges
    const int j = (s - P1) / g.S2, part = (s - P1) % g.S2, g0 = ng * part / g.S2, f0 = g.F2 * j / g.Pf;
    return {f0, g.F2 * (j + 1) / g.Pf - f0, g0, g0, ng * (part + 1) / g.S2};
  };
  auto next_tile = [&](bool second, FewRange& r, FewTile& t) -> bool {
    if (r.left <= 0) return false;
    t.f0 = r.f0;
    if (!second) {
      t.e = glist[r.g];
      // of the range in this group; the last two tiles alike, so that neither is narrow
      const int sh = gated ? 3 : 4, left = min(g.F1 - r.f0, r.left), step = 1 << sh;
      t.len = left >= 2 * g.rows1 ? g.rows1 : left > g.rows1 ? ((left >> 1) + step - 1) >> sh << sh : left;
      t.bi = (t.len - 1) >> sh;
      t.box = (t.bi + 1) << sh;
      r.left -= t.len;
      r.f0 += t.len;
      if (r.f0 == g.F1) {
        r.f0 = 0;
        ++r.g;
      }
      t.arows = gated ? 2 * t.box : t.box;
      t.rows = g.xrows;
      t.N = g.N;
      t.hs = g.hs1[t.bi];
      t.ns = g.ns1[t.bi];
    } else {
      if (r.g0 == r.g1) return false;
      t.e = glist[r.g];
      t.len = min(g.box2, r.left);
      t.box = t.arows = g.box2;
      if (++r.g == r.g1) {
        r.g = r.g0;
        r.f0 += t.len;
        r.left -= t.len;
      }
      const int m = __popcll(mask[t.e]);
      t.bi = box_of(m);
      t.rows = t.N = 16 << t.bi;      // both parts of y
      t.hs = g.hs2[t.bi];
      t.ns = g.ns2[t.bi];
    }
    return true;
  };

  if (warp == 0) {
    // ---------------- claims, and the weights' copies ----------------
    if (lane == 0) {
      const uint64_t policy = tc::policy_evict_first();
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        const int c = n == 0 ? claim : atomicAdd(g.ticket, 1), s = c < P1 + P2 ? c : -1;
        if (!tc::mbar_wait(&qempty[n % kFQueue], ((n / kFQueue) & 1) ^ 1, abort)) { ok = false; break; }
        queue[n % kFQueue] = s;
        tc::mbar_arrive(&qfull[n % kFQueue]);
        if (s < 0) break;
        const bool second = s >= P1;
        const int K = second ? g.K2 : g.K1, nh = (K + kFH - 1) / kFH;
        const bool chunks = K % kFH == 0;
        FewRange r = range_of(s);
        FewTile t;
        while (ok && next_tile(second, r, t)) {
          const int half = t.arows * 128, hs = t.hs;
          const CUtensorMap* map = second ? &maps.a2 : &maps.a[t.bi];
          const int ns = t.ns;
          for (int i = 0, h = first_stage(s, ns) * hs; i < ns; ++i, h = h + hs < nh ? h + hs : 0) {
            if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
            const int left = min(hs, nh - h), n_h = chunks ? (left + 1) & ~1 : left;
            tc::bar_arrive_expect_tx(full_u + 8 * slot, n_h * half);
            copy_weights(ring_u + slot * g.slot, half, map, chunks, h * kFH, n_h, t.f0, t.e, full_u + 8 * slot, policy);
            ++issued;
            if (++slot == g.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
      }
      if (!ok || *abort) wind_down(full, issued, g.stages);
    }
  } else if (warp == 2) {
    // ---------------- the rows' copies ----------------
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true, ready = false;
      for (uint32_t n = 0; ok; ++n) {
        const int s = take(n);
        if (s < 0) break;
        const bool second = s >= P1;
        if (second && !ready) {
          // every range of the first product has written its rows
          const long long t0 = clock64();
          for (uint32_t it = 1; ld_acquire_gpu(g.done) < P1; ++it) {
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
        const int K = second ? g.K2 : g.K1, nh = (K + kFH - 1) / kFH;
        const bool chunks = K % kFH == 0;
        FewRange r = range_of(s);
        FewTile t;
        while (ok && next_tile(second, r, t)) {
          // behind the stage's weights
          const int hs = t.hs, a_bytes = hs * t.arows * 128, half = t.rows * 128;
          const CUtensorMap* map = second ? &maps.y[t.bi] : &maps.x;
          const int r0 = second ? rowof[t.e] : 0;
          const int ns = t.ns;
          for (int i = 0, h = first_stage(s, ns) * hs; i < ns; ++i, h = h + hs < nh ? h + hs : 0) {
            if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
            const int left = min(hs, nh - h), n_h = chunks ? (left + 1) & ~1 : left;
            tc::bar_arrive_expect_tx(full_u + 8 * slot, n_h * half);
            if (second) copy_y(ring_u + slot * g.slot + a_bytes, half, map, chunks, h * kFH, n_h, r0, full_u + 8 * slot);
            else copy_rows(ring_u + slot * g.slot + a_bytes, half, map, chunks, h * kFH, n_h, r0, full_u + 8 * slot);
            ++issued;
            if (++slot == g.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        tc::mbar_arrive(&qempty[n % kFQueue]);
      }
      if (!ok || *abort) wind_down(full, issued, g.stages);
    }
  } else if (warp < 4 || warp >= 8) {
    // ---------------- MMAs ----------------
    const uint32_t wi = uni(warp), step = wi == 1 ? 0 : wi == 3 ? 1 : wi - 6;       // of every 64 of the reduction
    const uint64_t d0 = tc::smem_desc_sw128(ring_u);
    const uint32_t lo = uni((uint32_t)d0 + 2 * step), hi = uni((uint32_t)(d0 >> 32));
    const uint32_t tm = uni(tmem) + step * ncol, tmw = uni(tmem) + step * kFWide, bars = uni(full_u), accs = uni(tc::smem_u32(accfull));
    const uint32_t slot_step = (uint32_t)g.slot / 16;
    uint32_t slot = 0, at = lo, phase = 0, tiles = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const int s = (int)uni((uint32_t)take(n));      // one lane's answer, should a wait run out
      if (s < 0) break;
      const bool second = s >= P1;
      const int nh = ((second ? g.K2 : g.K1) + kFH - 1) / kFH;
      FewRange r = range_of(s);
      FewTile t;
      while (ok && next_tile(second, r, t)) {
        const uint32_t d = tiles & 1;
        if (!__all_sync(kFull, tc::mbar_wait(&accempty[d], ((tiles >> 1) & 1) ^ 1, abort))) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t a_step = uni(t.arows * 8), b_step = uni(t.rows * 8), hs = uni(t.hs), wide = uni(t.N);
        const uint32_t idesc = tc::idesc_16bit(a_step <= 64 * 8 ? 64 : kFM, wide, g.dtype == MOE_DT_BF16, 0, 0);
        // 128 columns: room for two accumulators a tile, so two of the warps issue, two steps each
        const bool narrow = wide < kFWide;
        const uint32_t dt = (narrow ? tm : tmw) + d * 4 * ncol;
        const uint32_t b_off = hs * a_step, ns = uni(t.ns);
        uint32_t acc = 0;
        for (uint32_t i = 0, h = uni(first_stage(s, ns)) * hs; i < ns; ++i) {
          if (!__all_sync(kFull, tc::bar_wait(bars + 8 * slot, phase, abort))) { ok = false; break; }
          tc::fence_after_sync();
          const uint32_t n_h = min(hs, (uint32_t)nh - h);
          uint32_t a = at, b = at + b_off;
          if (narrow) {
#pragma unroll 2
            for (uint32_t c = 0; c < n_h; ++c, a += a_step, b += b_step) {
              mma_one(dt, a, b, hi, idesc, acc);
              acc = 1;
            }
          } else if (step < 2) {
            a += 2 * step;              // steps 0 and 1, 2 and 3
            b += 2 * step;
            for (uint32_t c = 0; c < n_h; ++c, a += a_step, b += b_step) {
              mma_one(dt, a, b, hi, idesc, acc);
              mma_one(dt, a + 2, b + 2, hi, idesc, 1u);
              acc = 1;
            }
          }
          commit_one(bars + 8 * (kFMaxStages + slot));      // its `empty`
          h = h + hs < (uint32_t)nh ? h + hs : 0;
          at += slot_step;
          if (++slot == (uint32_t)g.stages) {
            slot = 0;
            at = lo;
            phase ^= 1;
          }
        }
        if (!ok) break;
        commit_one(accs + 8 * d);
        ++tiles;
      }
      if (lane == 0) tc::mbar_arrive(&qempty[n % kFQueue]);
    }
    // every MMA of this warp has completed once its `drain` fires
    __syncwarp();
    commit_one(uni(tc::smem_u32(&drain[step])));
    volatile int never = 0;
    tc::mbar_wait(&drain[step], 0, &never, 400000000ll);
    __syncwarp();
  } else {
    // ---------------- epilogue ----------------
    const int et = tid - 128, q = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    uint32_t tiles = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const int s = take(n);
      if (!epi_all<1, 128>(s >= 0)) break;
      const bool second = s >= P1;
      FewRange r = range_of(s);
      FewTile t;
      const int h0 = r.f0, nf = r.left;         // second: the range
      if (second && r.g0 == r.g1) {
        // no group, nothing to add
        if (g.S2 == 1) {
          for (int h = et; h < nf; h += 128)
            for (int i = 0; i < g.R; ++i) reinterpret_cast<uint16_t*>(g.out)[i * g.ldo + h0 + h] = 0;
        } else if (et < nf) {
          for (int i = 0; i < g.R; ++i) g.part[((int64_t)(s - P1) * g.R + i) * g.box2 + et] = 0.f;
        }
      }
      while (next_tile(second, r, t)) {
        const int d = tiles & 1;
        const bool got = tc::mbar_wait(&accfull[d], (tiles >> 1) & 1, abort);
        ++tiles;
        // the second product's warps meet at the end of the range only
        if (!(second ? __all_sync(kFull, got) != 0 : epi_all<1, 128>(got))) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t acc = lanes + d * 4 * ncol;
        auto release = [&] {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&accempty[d]);
        };
        unsigned long long rem = mask[t.e];
        const int m = __popcll(rem);
        // the thread's row of the tile: an MMA of 64 rows leaves sixteen to each warp's lanes
        const int row = t.arows > 64 ? et : lane < 16 ? q * 16 + lane : kFM;
        if (!second) {
          const int r0 = rowof[t.e];
          const bool all = g.N == 16;         // up to 16 tokens: all their columns at once, the group's own picked below
          const int step = all ? 16 : kFCols;
          for (int i0 = 0; i0 < m; i0 += step) {
            const int nc = min(step, m - i0);
            if (all) {
              uint32_t v[16];
              add_columns<16>(v, acc, ncol);
              if (row < kFM)
#pragma unroll
                for (int i = 0; i < 16; ++i) stage[i * kFM + row] = __uint_as_float(v[i]);
            } else {
              uint32_t v[kFCols][4];
#pragma unroll
              for (int i = 0; i < kFCols; ++i)
                if (i < nc) {
                  const uint32_t c = acc + next_bit(rem);
#pragma unroll
                  for (int j = 0; j < 4; ++j) tmem_ld1(c + j * ncol, v[i][j]);
                }
              tc::tmem_wait_ld();
              if (row < kFM)
#pragma unroll
                for (int i = 0; i < kFCols; ++i)
                  if (i < nc) stage[i * kFM + row] = add4(v[i]);
            }
            if (i0 + step >= m) release();
            epi_sync();
            // a thread's feature l of the tile, of every `skip`-th token
            const int l = et & (g.rows1 - 1), skip = 128 / g.rows1;
            unsigned long long cols = rem;                // all: the columns of the group's tokens
            if (et >= g.rows1) cols &= cols - 1;
            for (int i = et / g.rows1; i < nc; i += skip) {
              const int c = all ? __ffsll((long long)cols) - 1 : i, f = t.f0 + l;
              for (int j = 0; j < skip; ++j) cols &= cols - 1;
              if (l >= t.len) continue;
              float a = stage[c * kFM + l], u = gated ? stage[c * kFM + t.box + l] : 0.f;
              if (g.b1) {
                a += g.b1[(int64_t)t.e * 2 * g.F1 + f];
                u += g.b1[(int64_t)t.e * 2 * g.F1 + g.F1 + f];
              }
              const float y = wrow[r0 + i0 + i] * (gated ? act_two(a, u, g.act) : act_one(a, g.act.act));
              uint16_t* to = g.y + (int64_t)(r0 + i0 + i) * g.ldy + f;
              const uint16_t hi = E::from(y * (1.f / y_unit<E>()));
              *to = hi;
              // what the first part's rounding left (of an infinity nothing)
              to[(int64_t)(A + g.S * g.R) * g.ldy] = E::from(isinf(E::to(hi)) ? 0.f : y - E::to(hi) * y_unit<E>());
            }
            epi_sync();
          }
        } else {
          // a thread's feature is its own throughout: its sums need no barrier
          const bool mine = row < t.len;
          if (mine && t.e == glist[r.g0])
#pragma unroll 8
            for (int i = 0; i < g.R; ++i) sums[i * g.box2 + row] = 0.f;
          const uint8_t* tok = tokof + rowof[t.e];
          for (int i0 = 0; i0 < m; i0 += kFCols) {
            // the sums (of tokens that differ) are asked for together, and in front of the accumulators
            float* at[kFCols];
            float u[kFCols];
#pragma unroll
            for (int i = 0; i < kFCols; ++i) {
              at[i] = sums + tok[min(i0 + i, m - 1)] * g.box2 + (mine ? row : 0);
              u[i] = *at[i];
            }
            uint32_t v[kFCols], w[kFCols];          // of both parts of y
            if (t.bi < 3) {
              add_columns<kFCols>(v, acc + i0, ncol);
              add_columns<kFCols>(w, acc + (8 << t.bi) + i0, ncol);
            } else {
              add_columns<kFCols, 2>(v, acc + i0, kFWide);
              add_columns<kFCols, 2>(w, acc + kFWide / 2 + i0, kFWide);
            }
            if (i0 + kFCols >= m) release();
#pragma unroll
            for (int i = 0; i < kFCols; ++i)
              if (mine && i0 + i < m) *at[i] = u[i] + fmaf(__uint_as_float(v[i]), y_unit<E>(), __uint_as_float(w[i]));
          }
          if (mine && t.e == glist[r.g1 - 1])
#pragma unroll 8
            for (int i = 0; i < g.R; ++i) {
              const float v = sums[i * g.box2 + row];
              if (g.S2 == 1) reinterpret_cast<uint16_t*>(g.out)[i * g.ldo + t.f0 + row] = E::from(v);
              else g.part[((int64_t)(s - P1) * g.R + i) * g.box2 + row] = v;
            }
        }
      }
      if (second) ok = epi_all<1, 128>(ok);
      if (ok && !second) {
        // the range's rows are in memory, for the tensor copies of any CTA
        __threadfence();
        fence_proxy_async_global();
        epi_sync();
        if (et == 0) atom_add_acq_rel_gpu(g.done, 1);
      }
      if (ok && second && g.S2 > 1) {
        // whoever is the last of the features' parts adds them, in order
        const int j = (s - P1) / g.S2;
        __threadfence();
        epi_sync();
        if (et == 0) *last = atom_add_acq_rel_gpu(&g.joined[j], 1) == g.S2 - 1;
        epi_sync();
        if (*last) {
          __threadfence();
          // eight at a time, whose loads are all asked for before the first sum
          const float* set = g.part + (int64_t)j * g.S2 * g.R * g.box2;
          for (int i0 = et; i0 < g.R * nf; i0 += 8 * 128) {
            float v[8];
            int t[8], h[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int i = min(i0 + u * 128, g.R * nf - 1);
              t[u] = i / nf;
              h[u] = i - t[u] * nf;
              v[u] = __ldcg(set + t[u] * g.box2 + h[u]);
            }
            for (int w = 1; w < g.S2; ++w) {
              float p[8];
#pragma unroll
              for (int u = 0; u < 8; ++u) p[u] = __ldcg(set + (w * g.R + t[u]) * g.box2 + h[u]);
#pragma unroll
              for (int u = 0; u < 8; ++u) v[u] += p[u];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
              if (i0 + u * 128 < g.R * nf) reinterpret_cast<uint16_t*>(g.out)[t[u] * g.ldo + h0 + h[u]] = E::from(v[u]);
          }
        }
      }
      __syncwarp();
      if (warp == 4 && lane == 0) tc::mbar_arrive(&qempty[n % kFQueue]);
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort) set_status(g.status, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 8 * ncol);
  }
}

// ---- one dense product ------------------------------------------------------------
// Tiles of an equal range of features x N rows over the whole reduction, in even
// rounds over the SMs. A tile copies its features rounded up to 8 (a few rows of its
// neighbour, which the L2 serves); with weights on the M side one of 48 features
// costs 48 rows of copies, and what the MMA computes for the other lanes is not read.
// Measured, in us (in brackets the bytes at 6775 GB/s): 1 x 7168 x 2048 8.4 (4.3), 64 rows
// 11.0; 16 x 2 x 2048 x 7168 13.5 (8.7); what the bytes do not explain is launch, the
// first copies' latency and the epilogue behind the last MMA, one after the other. (Fixed
// tiles cut along the reduction, with their sums joined through memory: 13.9 and 86.)
constexpr int kDStages = 16;
constexpr int kDThreads = 448;
constexpr int kDCols = 16;            // columns an epilogue group takes at a time
constexpr int kDHead = 1024;          // barriers
constexpr int kDPad = 128 * 64;       // behind the ring, see launch_few_layer

template <typename E, bool GATED>
__global__ void __launch_bounds__(kDThreads, 1) k_few_linear(const FewArgs g, const __grid_constant__ FewMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* empty = full + kDStages;
  uint64_t* accfull = empty + kDStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + kFIssuers);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* stage = reinterpret_cast<float*>(base + kDHead);           // [2][kDCols][128]
  const int arows = (GATED ? 2 : 1) * g.rows1, a_half = arows * 128, b_half = g.N * 128;
  uint8_t* ring = base + g.head;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) {
      tc::mbar_init(&full[i], 2);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&accfull[i], g.issuers);
      tc::mbar_init(&accempty[i], 8);
    }
    for (int i = 0; i < kFIssuers; ++i) tc::mbar_init(&drain[i], 1);
    *abort = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.a[0]);
    tc::prefetch_tmap(&maps.x);
  }
  const uint32_t ncol = g.N <= 16 ? 16 : g.N <= 32 ? 32 : g.N <= 64 ? 64 : g.N <= 128 ? 128 : 256;
  uint32_t cols = 32;
  while (cols < 2 * g.issuers * ncol) cols *= 2;
  if (warp == 1) tc::tmem_alloc(tmem_slot, cols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_enter();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_u = tc::smem_u32(full), empty_u = tc::smem_u32(empty), ring_u = tc::smem_u32(ring);
  const int tiles = g.mt1 * g.nt, hs = g.hs, nh = (g.K1 + kFH - 1) / kFH, ns = (nh + hs - 1) / hs;

  if (warp == 0 || warp == 2) {
    // ---------------- copies: warp 0 weights, warp 2 rows ----------------
    if (lane == 0) {
      // weights that several row tiles read are worth keeping
      const uint64_t policy = g.nt > 1 ? tc::policy_evict_last() : tc::policy_evict_first();
      const bool chunks = g.K1 % kFH == 0;
      int slot = 0;
      uint32_t phase = 1, issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int f0 = (int)((int64_t)g.F1 * (t / g.nt) / g.mt1), r0 = t % g.nt * g.N;
        for (int i = 0, h = first_stage(t, ns) * hs; i < ns; ++i, h = h + hs < nh ? h + hs : 0) {
          if (!tc::bar_wait(empty_u + 8 * slot, phase, abort)) { ok = false; break; }
          const int left = min(hs, nh - h), n = chunks ? (left + 1) & ~1 : left;
          const uint32_t bar = full_u + 8 * slot, dst = ring_u + slot * g.slot;
          if (warp == 0) {
            tc::bar_arrive_expect_tx(bar, n * a_half);
            copy_weights(dst, a_half, &maps.a[0], chunks, h * kFH, n, f0, 0, bar, policy);
          } else {
            tc::bar_arrive_expect_tx(bar, n * b_half);
            copy_rows(dst + hs * a_half, b_half, &maps.x, chunks, h * kFH, n, r0, bar);
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
  } else if (warp < 4 || warp >= 12) {
    // ---------------- MMAs ----------------
    const uint32_t wi = uni(warp), who = wi < 4 ? wi >> 1 : wi - 10, many = (uint32_t)g.issuers;
    if (who < many) {
      const uint64_t d0 = tc::smem_desc_sw128(ring_u);
      const uint32_t lo = uni((uint32_t)d0), hi = uni((uint32_t)(d0 >> 32));
      const uint32_t tm = uni(tmem) + who * ncol, bars = uni(full_u), accs = uni(tc::smem_u32(accfull));
      const uint32_t idesc = tc::idesc_16bit(arows <= 64 ? 64 : kFM, g.N, g.dtype == MOE_DT_BF16, 0, 0);
      const uint32_t a_step = arows * 8, b_step = g.N * 8, b_off = hs * a_step, slot_step = (uint32_t)g.slot / 16;
      uint32_t slot = 0, at = lo, phase = 0, done = 0, turn = 0;      // turn: whose the next stage is
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++done) {
        const uint32_t d = done & 1;
        if (!__all_sync(kFull, tc::mbar_wait(&accempty[d], ((done >> 1) & 1) ^ 1, abort))) break;
        tc::fence_after_sync();
        const uint32_t dt = tm + d * many * ncol;
        uint32_t acc = 0;
        for (int i = 0, h = first_stage(t, ns) * hs; i < ns; ++i) {
          if (turn == who) {
            if (!__all_sync(kFull, tc::bar_wait(bars + 8 * slot, phase, abort))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t a = at, b = at + b_off;
            for (int c = min(hs, nh - h); c > 0; --c, a += a_step, b += b_step) {
              mma_four(dt, a, b, hi, idesc, acc);
              acc = 1;
            }
            commit_one(bars + 8 * (kDStages + slot));       // its `empty`
          }
          turn = turn + 1 == many ? 0 : turn + 1;
          h = h + hs < nh ? h + hs : 0;
          at += slot_step;
          if (++slot == (uint32_t)g.stages) {
            slot = 0;
            at = lo;
            phase ^= 1;
          }
        }
        if (ok) commit_one(accs + 8 * d);
      }
      // every MMA of this warp has completed once its `drain` fires
      __syncwarp();
      commit_one(uni(tc::smem_u32(&drain[who])));
      volatile int never = 0;
      tc::mbar_wait(&drain[who], 0, &never, 400000000ll);
      __syncwarp();
    }
  } else {
    // ---------------- epilogue ----------------
    // Two groups of four warps share a tile's columns, kDCols by kDCols. A lane
    // holds a feature; they go through shared memory, where the gate and up of a
    // gated tile meet, and are spread over all threads (each lane's own features
    // written from registers: 96 x 640 x 704 with GELU 7.7 us against 5.4).
    const int grp = (warp - 4) >> 2, q = warp & 3, et = (threadIdx.x - 128) & 127;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const int row = arows > 64 ? et : lane < 16 ? q * 16 + lane : kFM;       // the lane's row of the tile
    float* st = stage + grp * kDCols * kFM;
    const uint16_t* res = reinterpret_cast<const uint16_t*>(g.res);
    uint16_t *z = reinterpret_cast<uint16_t*>(g.z), *out = reinterpret_cast<uint16_t*>(g.out);
    auto bias = [&](int64_t f) {
      return !g.bias ? 0.f : g.wdtype == MOE_DT_F32 ? reinterpret_cast<const float*>(g.bias)[f]
                                                   : E::to(reinterpret_cast<const uint16_t*>(g.bias)[f]);
    };
    auto group_sync = [&] {
      __syncwarp();
      if (grp) asm volatile("bar.sync 2, 128;" ::: "memory");
      else asm volatile("bar.sync 1, 128;" ::: "memory");
    };
    uint32_t done = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++done) {
      const int d = done & 1, j = t / g.nt, r0 = t % g.nt * g.N, nr = min(g.N, g.R - r0);
      const int f0 = (int)((int64_t)g.F1 * j / g.mt1), nf = (int)((int64_t)g.F1 * (j + 1) / g.mt1) - f0;
      const uint32_t acc = lanes + d * g.issuers * ncol;
      // the accumulators of the tile's stages, from the first one's on, added
      auto columns = [&](int c, uint32_t (&v)[kDCols]) {
        uint32_t turn = done * (uint32_t)ns % (uint32_t)g.issuers;
        tc::tmem_ld16(acc + turn * ncol + c, v);
        tc::tmem_wait_ld();
        for (int w = 1; w < min(g.issuers, ns); ++w) {
          uint32_t u[kDCols];
          turn = turn + 1 == (uint32_t)g.issuers ? 0 : turn + 1;
          tc::tmem_ld16(acc + turn * ncol + c, u);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kDCols; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
        }
      };
      // thread: feature l of every `step`-th column
      const int step = 128 / g.lanes, l = et % g.lanes, i0 = et / g.lanes;
      const int64_t f = f0 + l;
      const float b0 = l < nf ? bias(f) : 0.f, b1 = GATED && l < nf ? bias((int64_t)g.F1 + f) : 0.f;
      constexpr int kMost = GATED ? kDCols / 2 : kDCols;      // columns of a chunk that are the thread's
      uint16_t rv[kMost];                                     // the next chunk's residual
      auto fetch = [&](int c) {
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
          const int i = c + i0 + k * step;
          rv[k] = res && k * step < kDCols && i < nr && l < nf ? res[(r0 + i) * g.ldr + f] : (uint16_t)0;
        }
      };
      fetch(grp * kDCols);
      const bool got = tc::mbar_wait(&accfull[d], (done >> 1) & 1, abort);
      if (!epi_all<3, 256>(got)) break;
      tc::fence_after_sync();
      for (int c = grp * kDCols; c < nr; c += 2 * kDCols) {
        const int n = min(kDCols, nr - c);
        uint32_t v[kDCols];
        columns(c, v);
        if (row < kFM)
#pragma unroll
          for (int i = 0; i < kDCols; ++i) st[i * kFM + row] = __uint_as_float(v[i]);
        group_sync();
        float add[kMost];
#pragma unroll
        for (int k = 0; k < kMost; ++k) add[k] = E::to(rv[k]);
        fetch(c + 2 * kDCols);
        if (l < nf) {
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int i = i0 + k * step;
            if (i >= n) break;
            const int64_t r = r0 + c + i;
            const float p = st[i * kFM + l] + b0;
            float y;
            if (z) z[r * g.ldz + f] = E::from(p);
            if constexpr (GATED) {
              const float u = st[i * kFM + g.rows1 + l] + b1;
              if (z) z[r * g.ldz + g.F1 + f] = E::from(u);
              y = act_two(p, u, g.act);
            } else {
              y = act_one(p, g.act.act);
            }
            out[r * g.ldo + f] = E::from(res ? y + add[k] : y);
          }
        }
        group_sync();
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
    tc::tmem_dealloc(tmem, cols);
  }
}

// ---- host -------------------------------------------------------------------------
// A ring of at most `most` stages, a multiple of its issuers, as many of those as can be:
// a slot is then always the same warp's, and one that waits for a use of a slot has
// itself seen the use before it (a barrier tells neighbouring uses apart only).
static void ring(FewArgs& g, int most, int issuers) {
  while (issuers > 1 && (most < issuers || most % issuers > 1)) --issuers;      // one stage may go unused
  g.issuers = issuers;
  g.stages = most / issuers * issuers;
}

// Weights [G][halves][rows][K]: boxes of 64 x box rows x halves, `depth` of them
// along K where K is a whole number of 64 (see copy_weights).
static bool map_weights(CUtensorMap* map, const void* w, int64_t K, int64_t rows, int halves, int64_t ld, int64_t G,
                        int64_t group, int box_rows, int depth) {
  const bool chunks = K % kFH == 0;
  const int64_t dims[5] = {chunks ? kFH : K, rows, halves, chunks ? K / kFH : 1, G};
  const int64_t strides[4] = {ld, halves > 1 ? rows * ld : ld, chunks ? kFH : ld, G > 1 ? group : ld};
  const int box[5] = {kFH, box_rows, halves, chunks ? depth : 1, 1};
  return make_tmap(map, w, 2, 5, dims, strides, box);
}
static bool map_rows(CUtensorMap* map, const void* x, int64_t K, int64_t rows, int64_t ld, int box_rows, int depth) {
  const bool chunks = K % kFH == 0;
  const int64_t dims[3] = {chunks ? kFH : K, rows, chunks ? K / kFH : 1}, strides[2] = {ld, chunks ? kFH : ld};
  const int box[3] = {kFH, box_rows, chunks ? depth : 1};
  return make_tmap(map, x, 2, 3, dims, strides, box);
}

static bool map_y(CUtensorMap* map, const void* y, int64_t K, int64_t rows, int64_t ld, int box_rows) {
  const bool chunks = K % kFH == 0;
  const int64_t dims[4] = {chunks ? kFH : K, rows, 2, chunks ? K / kFH : 1}, strides[3] = {ld, rows * ld, chunks ? kFH : ld};
  const int box[4] = {kFH, box_rows, 2, chunks ? 2 : 1};
  return make_tmap(map, y, 2, 4, dims, strides, box);
}

cudaError_t launch_few_layer(FewArgs g, const void* x, int64_t ldx, const void* w1, int64_t g1, int64_t ld1, const void* w2,
                             int64_t g2, int64_t ld2, cudaStream_t st) {
  const int G = g.E + g.S, A = g.R * g.k, halves = act_gated(g.act.act) ? 2 : 1;
  const int grid = std::min(device_sms(), kFewSms);
  g.N = (g.R + 15) & ~15;
  g.xrows = (g.R + 7) & ~7;
  g.rows1 = kFM / halves;
  int box_t = 8;                                    // rows of the second product's widest copy, of a part
  while (box_t < g.R) box_t *= 2;
  // y is a sum of two 16-bit numbers, side by side in the MMA's columns (its weights
  // are read once all the same): rounded to one, it leaves out 1.4 times as far off as out's own rounding, and where
  // few values are summed more (256 x 128, 1 token: 1.53); as two, 1.0. Four accumulators of up to 64 columns (groups of 32
  // tokens) fill tensor memory, two of 128 as well. In us, as one and as two, 64 tokens: x 2880 x 2880, 4 of 128 769, 775;
  // x 7168 x 2048, 8 of 64 849, 859; x 4096 x 512, 8 of 256 453, 450; with large groups, x 4096 x 14336, 2 of 8 426, 447; all
  // tokens on both of 2, 4096 x 2048 56.0, 61.4.
  g.ncol = 16;
  while (g.ncol < std::max(g.N, std::min(64, 2 * box_t))) g.ncol *= 2;
  // Bytes of a stage, of what stands in front of the ring, and its stages, by the
  // features of the second product's tiles. An MMA of 64 or 128 rows reads past the rows that were
  // copied, of A and of B (16 where 8 were): within the stage but for its last halves, where the tile is narrow.
  const int pad = 128 * 64;
  auto layout = [&](int box2) {
    const int head = kFBars + 16 * kFM * 4 + 4 * (g.R * box2 + 2) + 12 * G + 4 * std::min(G, A + g.S) + 5 * (A + g.S * g.R) + 8 * A;
    g.box2 = box2;
    g.slot = 2 * 128 * std::max(kFM + g.xrows, box2 + 2 * box_t);
    g.head = (head + 1023) / 1024 * 1024;
    g.stages = std::min(kFMaxStages, (kFSmem - 1024 - g.head - pad) / g.slot);
  };
  auto stages = [&](int rows, int64_t K, int& hs, int& ns) {
    hs = g.slot / (256 * rows) * 2;
    ns = (int)up(up(K, kFH), hs);
  };
  // The second product's ranges, with all groups or 1 / S2 of them, in cycles: a tile takes
  // its weights' bytes, the issue of its MMAs and stages, or that of its copies (two 64s of the reduction each where
  // those are whole), whichever is longest; a split costs the join; a ring of three stages instead of four a tenth.
  // Groups that some token chooses, when each chooses k at random. Measured, S2 = 1, 2 and 4, in us
  // behind the router: 16 tokens x 4096 x 512, 8 of 256 experts 239, 202, 204; 64 x 2048 x 1408, 6 of 64 221,
  // 180, 188; 16 x 2880 x 2880, 4 of 128 403, 373, 380; 64 x 7168 x 2048, 8 of 64 853, 869, -; 64 x 1024 x 256, 8 of
  // 64 76, 55, 45; 1 x 256 x 128, 2 of 8 11.7, 14.2, 15.0.
  const double touched = g.E * (1 - std::pow(1 - (double)g.k / g.E, g.R)) + g.S;
  const double nh = (double)up(g.K2, kFH), copies = g.K2 % kFH ? nh : nh / 2;
  int rows = 8;                                     // of a tile's copies
  while (rows < box_t && rows * touched < (double)A + g.S * g.R) rows *= 2;
  double least = 1e300;
  int most = 1;
  for (int S2 = 1; S2 <= 4; S2 *= 2) {
    const int Pf = (int)std::min<int64_t>(grid / S2, up(g.F2, kFLeast)), f = (int)up(g.F2, Pf);
    if (S2 > 1 && f > kFM) break;
    layout(std::min(kFM, (f + 7) & ~7));
    if (g.stages < 2) {           // beside the tables of 2000 experts; narrower tiles for a split range there are not
      if (S2 > 1) break;
      layout(64);
    }
    int hs, ns;
    stages(g.box2 + 2 * rows, g.K2, hs, ns);
    const double tile = std::max({nh * 128 * std::min((double)g.F2 / Pf, (double)kFM) / 23.5, 600 + 90 * nh + 300 * ns, 150 * copies + 200 * ns});
    const double cost = touched / S2 * tile * up(f, kFM) * (g.stages < 4 ? 1.1 : 1.) + (S2 > 1 ? 3000 + 1000 * S2 + 6. * g.R * f : 0);
    if (cost < least) {
      least = cost;
      g.S2 = S2; g.Pf = Pf;
      most = g.box2;
    }
  }
  layout(most);
  for (int i = 0; i < 8; ++i) stages(16 * (i + 1) + g.xrows, g.K1, g.hs1[i], g.ns1[i]);      // halves * step * (i + 1) rows
  for (int i = 0; i < 4; ++i) stages(g.box2 + 2 * std::min(8 << i, box_t), g.K2, g.hs2[i], g.ns2[i]);
  const int smem = 1024 + g.head + g.stages * g.slot + pad;
  FewMaps maps;
  for (int i = 0; i < 8; ++i)
    if (!map_weights(&maps.a[i], w1, g.K1, g.F1, halves, ld1, G, g1, g.rows1 / 8 * (i + 1), 2)) return cudaErrorInvalidValue;
  for (int i = 0; i < 4; ++i)
    if (!map_y(&maps.y[i], g.y, g.K2, (int64_t)g.R * (g.k + g.S), g.ldy, 8 << i)) return cudaErrorInvalidValue;
  if (!map_weights(&maps.a2, w2, g.K2, g.F2, 1, ld2, G, g2, g.box2, 2) || !map_rows(&maps.x, x, g.K1, g.R, ldx, g.xrows, 2))
    return cudaErrorInvalidValue;
  const auto kernel = g.dtype == MOE_DT_BF16 ? k_few_layer<Bf16> : k_few_layer<F16>;
  static std::atomic<bool> done[2][kMaxDevices] = {};
  const cudaError_t e = set_smem_once((const void*)kernel, kFSmem, done[g.dtype == MOE_DT_BF16]);
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(kernel, dim3(grid), dim3(kFThreads), smem, st, g, maps);
}

template <typename E, bool GATED>
static cudaError_t launch_linear(FewArgs& g, const FewMaps& maps, int grid, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices] = {};
  const cudaError_t e = set_smem_once((const void*)k_few_linear<E, GATED>, kFSmem, done);
  if (e != cudaSuccess) return e;
  const int half = 128 * ((GATED ? 2 : 1) * g.rows1 + g.N);
  g.hs = std::min(std::max(1, 32768 / (2 * half)) * 2, stage_halves(g.K1));
  g.slot = g.hs * half;
  g.head = (kDHead + 2 * kDCols * kFM * 4 + 1023) / 1024 * 1024;
  // no more issuers than tensor memory has room for accumulators; wide MMAs need fewer
  ring(g, std::min(kDStages, (kFSmem - 1024 - g.head - kDPad) / g.slot), g.N <= 64 ? kFIssuers : g.N <= 128 ? 2 : 1);
  g.lanes = g.rows1 <= 16 ? 16 : g.rows1 <= 32 ? 32 : g.rows1 <= 64 ? 64 : 128;
  note_launch();
  return launch_pdl(k_few_linear<E, GATED>, dim3(grid), dim3(kDThreads), 1024 + g.head + g.stages * g.slot + kDPad, st, g, maps);
}

cudaError_t launch_few_linear(FewArgs g, const void* x, int64_t ldx, const void* w, int64_t ldw, cudaStream_t st) {
  const bool gated = act_gated(g.act.act);
  const int halves = gated ? 2 : 1, sms = device_sms();
  // the tiles with the least to copy: rounds over the SMs times their rows of both
  // operands, and a fixed cost of a round
  int64_t least = INT64_MAX;
  for (int nt = (int)up(g.R, 256); nt <= up(g.R, 16); ++nt) {
    const int n = (int)(up(up(g.R, nt), 16) * 16);
    if (up(g.R, n) != nt || n > 240) continue;
    const int64_t most = up(g.F1, 8);             // ranges
    for (int64_t rounds = std::max<int64_t>(1, up(up(g.F1, kFM / halves) * nt, sms));; ++rounds) {
      const int64_t mt = std::min(most, std::max<int64_t>(1, rounds * sms / nt)), box = up(up(g.F1, mt), 8) * 8;
      // three stages at least
      if (box * halves <= kFM && box * halves + n <= 256) {
        const int64_t cost = up(mt * nt, sms) * (box * halves + n + 16);
        if (cost < least) {
          least = cost;
          g.rows1 = (int)box; g.N = n; g.nt = nt; g.mt1 = (int)mt;
        }
        if (box * halves + n <= 96) break;        // smaller tiles only add rounds
      }
      if (mt == most) break;
    }
  }
  FewMaps maps = {};
  if (!map_weights(&maps.a[0], w, g.K1, g.F1, halves, ldw, 1, 0, g.rows1, 2) || !map_rows(&maps.x, x, g.K1, g.R, ldx, g.N, 2))
    return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>((int64_t)g.mt1 * g.nt, sms);
  if (gated)
    return g.dtype == MOE_DT_BF16 ? launch_linear<Bf16, true>(g, maps, grid, st) : launch_linear<F16, true>(g, maps, grid, st);
  return g.dtype == MOE_DT_BF16 ? launch_linear<Bf16, false>(g, maps, grid, st) : launch_linear<F16, false>(g, maps, grid, st);
}

}  // namespace moe
