// The routed layer for a few tokens with experts in 16 bits: router, top-k, both
// products with the activation between them, combine.
#include "ops.cuh"

namespace moe {

static int64_t al256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: y [T (k + S)][I] 16-bit rows, by token and slot.
int64_t layer16_ws_bytes(int T, int H, int I, int E, int k, int S) {
  return al256((int64_t)T * (k + S) * I * 2);
}

// One CTA routes one token.
template <typename E>
__global__ void __launch_bounds__(256) k_l16_route(const Layer16Args a) {
  __shared__ float lg[2048];
  pdl_enter();
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

// The expert and weight of slot j of token t; false: nothing to add.
__device__ __forceinline__ bool slot_of(const Layer16Args& a, int t, int j, int& e, float& w) {
  if (j >= a.k) { e = a.E + j - a.k; w = 1.f; return true; }
  e = a.ids[t * a.k + j];
  w = a.w[t * a.k + j];
  if (e < 0 || e >= a.E) { set_status(a.status, MOE_DEV_BAD_EXPERT_ID); return false; }
  return w != 0.f;
}
template <typename E>
__device__ __forceinline__ float dot(const uint16_t* a, const uint16_t* b, int n, int lane) {
  float s = 0.f;
  for (int i = lane; i < n; i += 32) s = fmaf(E::to(a[i]), E::to(b[i]), s);
  return warp_sum(s);
}

// y[t, j, i] of one token and slot: a warp a feature.
template <typename E>
__global__ void __launch_bounds__(256) k_l16_w1(const Layer16Args a) {
  pdl_enter();
  const int kp = a.k + a.S, t = blockIdx.y / kp, j = blockIdx.y % kp, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  int e;
  float w;
  if (i >= a.I || !slot_of(a, t, j, e, w)) return;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + t * a.ldx;
  const uint16_t* w1 = reinterpret_cast<const uint16_t*>(a.w1) + e * a.g1;
  float g = dot<E>(x, w1 + i * a.ld1, a.H, lane), y;
  if (act_gated(a.act.act)) {
    float u = dot<E>(x, w1 + (int64_t)(a.I + i) * a.ld1, a.H, lane);
    if (a.b1) { g += a.b1[(int64_t)e * 2 * a.I + i]; u += a.b1[(int64_t)e * 2 * a.I + a.I + i]; }
    y = act_two(g, u, a.act);
  } else {
    y = act_one(g, a.act.act);
  }
  if (lane == 0) reinterpret_cast<uint16_t*>(a.ws)[(int64_t)blockIdx.y * a.I + i] = E::from(w * y);
}

// out[t, h] over the token's slots, in slot order: a warp a column.
template <typename E>
__global__ void __launch_bounds__(256) k_l16_w2(const Layer16Args a) {
  pdl_enter();
  const int kp = a.k + a.S, t = blockIdx.y, lane = threadIdx.x & 31, h = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (h >= a.H) return;
  float s = 0.f;
  for (int j = 0; j < kp; ++j) {
    int e;
    float w;
    if (!slot_of(a, t, j, e, w)) continue;
    s += dot<E>(reinterpret_cast<const uint16_t*>(a.ws) + (int64_t)(t * kp + j) * a.I,
                reinterpret_cast<const uint16_t*>(a.w2) + e * a.g2 + h * a.ld2, a.I, lane);
  }
  if (lane == 0) reinterpret_cast<uint16_t*>(a.out)[t * a.ldo + h] = E::from(s);
}

template <typename E>
static cudaError_t launch_typed(const Layer16Args& a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.W_r || a.logits) {
    note_launch();
    if ((e = launch_pdl(k_l16_route<E>, dim3(a.T), dim3(256), 0, st, a)) != cudaSuccess) return e;
  }
  note_launch();
  if ((e = launch_pdl(k_l16_w1<E>, dim3((a.I + 7) / 8, a.T * (a.k + a.S)), dim3(256), 0, st, a)) != cudaSuccess) return e;
  note_launch();
  return launch_pdl(k_l16_w2<E>, dim3((a.H + 7) / 8, a.T), dim3(256), 0, st, a);
}

cudaError_t launch_layer16(const Layer16Args& a, cudaStream_t st) {
  return a.dtype == MOE_DT_BF16 ? launch_typed<Bf16>(a, st) : launch_typed<F16>(a, st);
}

}  // namespace moe
