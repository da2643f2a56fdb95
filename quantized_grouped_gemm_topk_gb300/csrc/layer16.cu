// The routed layer for a few tokens with experts in 16 bits: router, top-k, both
// products with the activation between them, combine.
#include "few16.cuh"

namespace moe {

static int64_t al256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: the counters, y [T (k + S)][I] 16-bit and z [T (k + S)][H] fp32 rows
// by group, partial sums.
struct Layer16Ws {
  int64_t ldy, ldz, counters, y, z, part, bytes;
};
static Layer16Ws layer16_ws(int T, int H, int I, int E, int k, int S) {
  Layer16Ws w;
  const int64_t rows = (int64_t)T * (k + S);
  w.ldy = (I + 7) / 8 * 8;
  w.ldz = (H + 127) / 128 * 128;
  w.counters = 16 + kFewShares + w.ldz / 128;
  w.y = al256(w.counters * 4);
  w.z = w.y + al256(rows * w.ldy * 2);
  w.part = w.z + al256(rows * w.ldz * 4);
  w.bytes = w.part + few_part_bytes(T);
  return w;
}
int64_t layer16_ws_bytes(int T, int H, int I, int E, int k, int S) { return layer16_ws(T, H, I, E, k, S).bytes; }

// One CTA routes one token.
template <typename E>
__global__ void __launch_bounds__(256) k_l16_route(const Layer16Args a, int64_t counters) {
  __shared__ float lg[2048];
  pdl_enter();
  // the products' counters, which the kernel behind this one starts from
  if (blockIdx.x == 0)
    for (int64_t i = threadIdx.x; i < counters; i += 256) reinterpret_cast<int32_t*>(a.ws)[i] = 0;
  if (!a.W_r && !a.logits) return;
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + t * a.ldx;
  for (int e = threadIdx.x; e < a.E; e += 256) {
    float v = 0.f;
    if (a.W_r) for (int h = 0; h < a.H; ++h) v = fmaf(E::to(x[h]), a.W_r[(int64_t)h * a.E + e], v);
    else v = a.logits[(int64_t)t * a.E + e];
    if (v != v) set_status(a.status, MOE_DEV_NAN_LOGIT);
    lg[e] = v != v ? -INFINITY : v;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  float sel = 0.f;
  int id = 0;
  for (int j = 0; j < a.k; ++j) {
    float best = 0.f;
    int at = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32) {
      const float v = lg[e];
      if (v == v && (at == 0x7fffffff || v > best)) { best = v; at = e; }     // a taken one is NaN
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float v = __shfl_xor_sync(kFull, best, o);
      const int i = __shfl_xor_sync(kFull, at, o);
      if (i != 0x7fffffff && (at == 0x7fffffff || v > best || (v == best && i < at))) { best = v; at = i; }
    }
    if (lane == 0) lg[at] = __int_as_float(0x7fffffff);
    __syncwarp();
    if (lane == j) { sel = best; id = at; }
  }
  const float m = __shfl_sync(kFull, sel, 0);
  const float p = lane < a.k && m != -INFINITY ? expf(sel - m) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < a.k; ++j) sum += __shfl_sync(kFull, p, j);
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.w[t * a.k + lane] = m != -INFINITY ? p / sum * a.rs : 0.f;
  }
}

cudaError_t launch_layer16(const Layer16Args& a, cudaStream_t st) {
  const Layer16Ws w = layer16_ws(a.T, a.H, a.I, a.E, a.k, a.S);
  note_launch();
  cudaError_t e = launch_pdl(a.dtype == MOE_DT_BF16 ? k_l16_route<Bf16> : k_l16_route<F16>, dim3(a.T), dim3(256), 0, st, a,
                             w.counters);
  if (e != cudaSuccess) return e;
  FewArgs f = {};
  f.R = a.T; f.K1 = a.H; f.F1 = a.I; f.K2 = a.I; f.F2 = a.H; f.act = a.act; f.dtype = a.dtype; f.status = a.status;
  f.E = a.E; f.k = a.k; f.S = a.S; f.ids = a.ids; f.wts = a.w; f.b1 = a.b1;
  f.y = reinterpret_cast<uint16_t*>(a.ws + w.y); f.ldy = w.ldy;
  f.zrow = reinterpret_cast<float*>(a.ws + w.z); f.ldz32 = w.ldz;
  f.part = reinterpret_cast<float*>(a.ws + w.part);
  f.ticket = reinterpret_cast<int32_t*>(a.ws);
  f.done = f.ticket + 8;
  f.split = f.ticket + 16;
  f.split2 = f.split + kFewShares;
  f.out = a.out; f.ldo = a.ldo;
  return launch_few_layer(f, a.x, a.ldx, a.w1, a.g1, a.ld1, a.w2, a.g2, a.ld2, st);
}

}  // namespace moe
