// Blocks of 128 columns of 16-bit rows in registers, and their E4M3 codes:
// shared by the quantisers and the activation checkpoints.
#pragma once
#include "ops.cuh"

namespace moe {

// A block's 128 columns belong to eight lanes, sixteen to a lane: columns
// 8 l .. 8 l + 7 and 64 + 8 l .. . Sixteen, so that a block's fixed work (the
// scales' divisions, shuffles, addresses) is spread over more elements. Held
// as words of two 16-bit elements (four codes). These four where every eight
// start on a 16-byte (codes: 8-byte) boundary and rows are of a multiple of
// eight; the ones by way of shared memory below at any alignment. Columns past
// the block's n read as zeros and are not written.
__device__ __forceinline__ void load16(uint32_t (&w)[8], const uint16_t* p, int l, int n) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = 64 * k + 8 * l;
    const uint4 u = c < n ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0u, 0u, 0u, 0u);
    w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
  }
}
template <typename E>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  return make_float2(E::to((uint16_t)(w & 0xffffu)), E::to((uint16_t)(w >> 16)));
}
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&w)[8], int l, int n) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = 64 * k + 8 * l;
    if (c < n) *reinterpret_cast<uint4*>(p + c) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}
// A block at any alignment by way of shared memory: each lane's columns go to
// `buf` (the quarter-warp's own, kStageBytes) at the block's place in its
// 16-byte units, and after a __syncwarp the lanes store whole units from there.
// Their own columns would leave in words and halves of a 32-byte sector each.
constexpr int kStageBytes = 256 + 16;
__device__ __forceinline__ void stage16(uint8_t* buf, const uint16_t* p, const uint32_t (&w)[8], int l) {
  const int off = (int)((uintptr_t)p & 15);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t v[4] = {w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
    store_inner<2>(buf + off + 128 * k + 16 * l, v);
  }
}
__device__ __forceinline__ void store_staged(uint16_t* p, const uint8_t* buf, int l, int n) {
  const int off = (int)((uintptr_t)p & 15), end = off + 2 * n;
  uint8_t* base = reinterpret_cast<uint8_t*>(p) - off;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int at = 16 * (8 * k + l);
    if (at >= off && at + 16 <= end) *reinterpret_cast<uint4*>(base + at) = *reinterpret_cast<const uint4*>(buf + at);
  }
  // what lies in the first and the last unit besides: an element a lane
  const int e = 2 * l, first = min(16, end), last = end & ~15;
  if (off && e >= off && e < first)
    *reinterpret_cast<uint16_t*>(base + e) = *reinterpret_cast<const uint16_t*>(buf + e);
  if ((!off || last) && last + e < end)
    *reinterpret_cast<uint16_t*>(base + last + e) = *reinterpret_cast<const uint16_t*>(buf + last + e);
}
__device__ __forceinline__ void load_codes(uint32_t (&w)[4], const uint8_t* q, int l, int n) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = 64 * k + 8 * l;
    const uint2 v = c < n ? *reinterpret_cast<const uint2*>(q + c) : make_uint2(0u, 0u);
    w[2 * k] = v.x;
    w[2 * k + 1] = v.y;
  }
}
__device__ __forceinline__ void store_codes(uint8_t* q, const uint32_t (&w)[4], int l, int n) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = 64 * k + 8 * l;
    if (c < n) *reinterpret_cast<uint2*>(q + c) = make_uint2(w[2 * k], w[2 * k + 1]);
  }
}
// The codes of a block at any address by way of shared memory: eight at a time
// to their columns' place in `buf` (kCodeBytes), after a __syncwarp whole units
// of the row from there, what is left at the block's ends byte by byte.
constexpr int kCodeBytes = 128 + 16;
__device__ __forceinline__ void stage_codes(uint8_t* buf, const uint32_t (&w)[4], int l) {
#pragma unroll
  for (int k = 0; k < 2; ++k) *reinterpret_cast<uint2*>(buf + 64 * k + 8 * l) = make_uint2(w[2 * k], w[2 * k + 1]);
}
__device__ __forceinline__ void store_staged_codes(uint8_t* q, const uint8_t* buf, int l, int n) {
  const int off = (int)((uintptr_t)q & 15), at = 16 * l - off;
  if (at >= 0 && at + 16 <= n) {
    const uint8_t* p = buf + (at & ~15);
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
    uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, r[4];
    shift_units<1, 16>(r, u, at & 15);
    *reinterpret_cast<uint4*>(q + at) = make_uint4(r[0], r[1], r[2], r[3]);
  }
  const int last = ((off + n) & ~15) - off;
#pragma unroll
  for (int e = l; e < 16; e += 8) {
    if (off && e < min(n, 16 - off)) q[e] = buf[e];
    if (last >= 0 && last + e < n) q[last + e] = buf[last + e];
  }
}

// Columns [c, c + 128) of a row of `n` elements of ES bytes, at any alignment,
// on their way to shared memory (asynchronous copies, to be committed and
// waited for): the 16-byte units that hold them, U = 8 ES + 1 of them at `buf`.
// Bytes past the block or the row become zeros and are not read; a first unit that
// begins before `base`, the tensor's first byte, is read byte by byte.
template <int ES>
__device__ __forceinline__ void fetch_block(uint8_t* buf, const uint8_t* row, int c, int n, const uint8_t* base,
                                            int l) {
  const uint8_t* p = row + (int64_t)c * ES;
  const int off = (int)((uintptr_t)p & 15);
  const uint8_t* at = p - off + 16 * l;
  const int left = min(n - c, kQBlock) * ES + off - 16 * l;     // bytes of the block from `at`
  auto unit = [&](int u) {
    const int bytes = min(16, max(0, left - 16 * u));
    cp_async16(buf + 16 * (l + u), bytes ? at + 16 * u : base - ((uintptr_t)base & 15), bytes);
  };
  if (at >= base) {
    unit(0);
  } else {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) buf[16 * l + i] = at + i >= base && i < left ? at[i] : 0;
  }
  if (ES == 2) unit(8);
  if (l == 0) unit(8 * ES);
}
// The lane's sixteen elements of a block in shared memory; off: the place of
// its first byte in the first unit.
__device__ __forceinline__ void read16(uint32_t (&w)[8], const uint8_t* buf, int off, int l) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 a = *reinterpret_cast<const uint4*>(buf + 128 * k + 16 * l);
    const uint4 b = *reinterpret_cast<const uint4*>(buf + 128 * k + 16 * l + 16);
    uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, r[4];
    shift_units<2, 16>(r, u, off);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * k + i] = r[i];
  }
}
__device__ __forceinline__ void read_codes(uint32_t (&w)[4], const uint8_t* buf, int off, int l) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint8_t* p = buf + (off & 8) + 64 * k + 8 * l;
    const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + 8);
    uint32_t u[4] = {a.x, a.y, b.x, b.y}, r[2];
    shift_units<1, 8>(r, u, off & 7);
    w[2 * k] = r[0];
    w[2 * k + 1] = r[1];
  }
}

// Magnitude bits (16-bit elements without their sign order as integers:
// finite < infinity < NaN) of the largest of the lane's sixteen.
__device__ __forceinline__ uint32_t mag_bits(const uint32_t (&w)[8]) {
  constexpr uint32_t k = 0x7fff7fffu;
  uint32_t m = w[0] & k;
#pragma unroll
  for (int j = 1; j < 8; ++j) m = __vmaxu2(m, w[j] & k);
  return max(m & 0xffffu, m >> 16);
}
// Codes of sixteen values at 1 / inv; FIN: without the test for infinities.
template <typename E, bool FIN>
__device__ __forceinline__ void codes16(uint32_t (&c)[4], const uint32_t (&w)[8], float inv) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = pair_of<E>(w[2 * j]), b = pair_of<E>(w[2 * j + 1]);
    const uint32_t lo = FIN ? f32x2_to_e4m3x2(a.x * inv, a.y * inv)
                            : f32x2_to_e4m3x2(code_arg(a.x, inv), code_arg(a.y, inv));
    const uint32_t hi = FIN ? f32x2_to_e4m3x2(b.x * inv, b.y * inv)
                            : f32x2_to_e4m3x2(code_arg(b.x, inv), code_arg(b.y, inv));
    c[j] = lo | (hi << 16);
  }
}
// The block's scale where some element is an infinity or NaN: the largest of
// the finite ones, over the eight lanes.
template <typename E>
__device__ __forceinline__ float finite_scale(const uint32_t (&w)[8], unsigned lanes) {
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 a = pair_of<E>(w[j]);
    am = fmaxf(am, fmaxf(finite_mag(a.x), finite_mag(a.y)));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(lanes, am, o));
  return block_scale(am);
}

// Quarter-warps of a CTA's `all` (a power of two) for a row of C columns: the
// most that leave at most a tenth of them idle in the row's last round.
inline int quarters_a_row(int C, int all) {
  const int nb = (C + kQBlock - 1) / kQBlock;
  int q = all;
  while (q > 1 && 10 * ((nb + q - 1) / q * q) > 11 * nb) q /= 2;
  return q;
}

}  // namespace moe
