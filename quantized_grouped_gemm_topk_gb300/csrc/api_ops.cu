// C entry points of the training-side operators: argument checks and
// launches. As the layer's calls, these only enqueue kernels on the caller's
// stream: no allocation, no synchronisation (moe_mm_read_status excepted).
#include "ops.cuh"

using namespace moe;

namespace {

constexpr size_t kStatusBytes = 256;   // the status word's block in a products' workspace; all behind it is scratch
constexpr size_t kArriveAt = 128;      // in it, the few tokens' layer's counters

bool is16(int dt) { return dt == MOE_DT_BF16 || dt == MOE_DT_F16; }
bool is_float(int dt) { return is16(dt) || dt == MOE_DT_F32; }
size_t size_of(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// non-NULL and aligned to n bytes
bool have(const void* p, size_t n) { return p && aligned(p, n); }
bool maybe(const void* p, size_t n) { return aligned(p, n); }
moe_status_t done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool act_ok(int act, float limit) {
  return act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU || act == MOE_ACT_SRELU ||
         (act == MOE_ACT_SWIGLU_CLAMP && limit > 0.f);
}
int64_t blocks_of(int64_t n) { return (n + kQBlock - 1) / kQBlock; }

// Sizes up to 2^30 leave room to round up to whole tiles and blocks, and to
// step past the end, in 32 bits.
constexpr int kMost = 1 << 30;
bool width_ok(int n) { return n >= 1 && n <= kMost; }
bool mm_sizes_ok(int R, int N, int K, int G) {
  return R >= 0 && R <= kMost && width_ok(N) && width_ok(K) && G >= 1 && G <= 2048;
}

// Elements from the first to the last of a rows x cols matrix with row stride
// ld: the least a group's stride may be.
int64_t span(int rows, int cols, int64_t ld) { return (int64_t)(rows - 1) * ld + cols; }

// Common checks of a product's sizes and workspace.
moe_status_t mm_check(int kind, int R, int N, int K, int G, const int32_t* offsets, void* ws, size_t ws_bytes) {
  if (!mm_sizes_ok(R, N, K, G)) return MOE_ERR_INVALID_ARG;
  if (!maybe(offsets, 4) || (!offsets && (G != 1 || kind != MOE_MM_FP8))) return MOE_ERR_INVALID_ARG;
  if (!have(ws, 16)) return MOE_ERR_INVALID_ARG;
  const int S = mm_splits(kind, R, N, K, G);
  const size_t outs = kind == MOE_MM_WGRAD ? (size_t)G * N * K : (size_t)R * N;
  return ws_bytes < kStatusBytes + (S > 1 ? outs * 4 * S : 0) ? MOE_ERR_WORKSPACE : MOE_OK;
}
void mm_workspace(MmArgs& a, int kind, void* ws) {
  a.status = reinterpret_cast<int32_t*>(ws);
  a.S = mm_splits(kind, a.R, a.N, a.K, a.G);
  a.part = a.S > 1 ? reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + kStatusBytes) : nullptr;
}

// The dense products' activations, and sizes (a gated one has 2 N weight rows).
bool linear_act_ok(int act, float limit) {
  return act_ok(act, limit) || act == MOE_ACT_NONE || act == MOE_ACT_GELU || act == MOE_ACT_SILU;
}
bool linear_sizes_ok(int R, int N, int K, int act) {
  return R >= 0 && R <= kMost && N >= 1 && N <= (act_gated(act) ? kMost / 2 : kMost) && width_ok(K);
}
void linear_workspace(LinearArgs& a, void* ws) {
  a.status = reinterpret_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + kStatusBytes);
}
bool layer16_sizes_ok(int T, int H, int I, int E, int k, int S) {
  constexpr int kWide = 1 << 20;
  return T >= 0 && H >= 1 && H <= kWide && I >= 1 && I <= kWide && (S == 0 || S == 1) && E >= 1 && E <= 2048 - S &&
         k >= 1 && k <= E && k + S <= 32;
}

}  // namespace

extern "C" {

moe_status_t moe_layer_norm_workspace_size(int64_t T, int H, size_t* bytes) {
  if (T < 0 || !width_ok(H) || !bytes) return MOE_ERR_INVALID_ARG;
  *bytes = (size_t)std::min<int64_t>(T, kNormMaxParts) * 2 * (size_t)H * 4;
  return MOE_OK;
}

moe_status_t moe_layer_norm_forward(const void* x, int64_t ldx, const void* gamma, const void* beta, float eps,
                                    int64_t T, int H, int dtype, int wdtype, void* y, int64_t ldy, float* mean,
                                    float* rstd, void* stream) {
  if (T < 0 || !width_ok(H) || !is_float(dtype) || (wdtype != MOE_DT_F32 && wdtype != dtype)) return MOE_ERR_INVALID_ARG;
  if (ldx < H || ldy < H || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  const size_t e = size_of(dtype), we = size_of(wdtype);
  if (!maybe(gamma, we) || !maybe(beta, we) || !maybe(mean, 4) || !maybe(rstd, 4)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  if (T == 0) return MOE_OK;
  if (!have(x, e) || !have(y, e)) return MOE_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = x; a.ldx = ldx; a.gamma = gamma; a.beta = beta; a.eps = eps; a.T = T; a.H = H;
  a.dtype = dtype; a.wdtype = wdtype; a.out = y; a.ldo = ldy; a.mean = mean; a.rstd = rstd;
  return done(launch_norm_fwd(a, (cudaStream_t)stream));
}

moe_status_t moe_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* gamma,
                                     const float* mean, const float* rstd, int64_t T, int H, int dtype, int wdtype,
                                     void* dx, int64_t lddx, void* dgamma, void* dbeta, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (T < 0 || !width_ok(H) || !is_float(dtype) || (wdtype != MOE_DT_F32 && wdtype != dtype)) return MOE_ERR_INVALID_ARG;
  if (lddy < H || ldx < H || lddx < H) return MOE_ERR_INVALID_ARG;
  const size_t e = size_of(dtype), we = size_of(wdtype);
  if (!maybe(gamma, we) || !maybe(dgamma, we) || !maybe(dbeta, we)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  reset_launch_count();
  if (T == 0) {     // the sums over no rows
    if (dgamma && cudaMemsetAsync(dgamma, 0, (size_t)H * we, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbeta && cudaMemsetAsync(dbeta, 0, (size_t)H * we, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!have(dy, e) || !have(x, e) || !have(dx, e) || !have(mean, 4) || !have(rstd, 4)) return MOE_ERR_INVALID_ARG;
  if (dgamma || dbeta) {
    size_t need = 0;
    const moe_status_t s = moe_layer_norm_workspace_size(T, H, &need);
    if (s != MOE_OK) return s;
    if (!have(ws, 16)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  }
  NormArgs a = {};
  a.x = x; a.ldx = ldx; a.dy = dy; a.lddy = lddy; a.gamma = gamma; a.T = T; a.H = H;
  a.dtype = dtype; a.wdtype = wdtype; a.out = dx; a.ldo = lddx;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.dgamma = dgamma; a.dbeta = dbeta; a.part = reinterpret_cast<float*>(ws);
  return done(launch_norm_bwd(a, st));
}

moe_status_t moe_act_ckpt_forward(const void* h, int64_t ldh, const float* w_row, int64_t R, int I, int dtype,
                                  int act, float alpha, float limit, void* y, int64_t ldy, uint8_t* q, int64_t ldq,
                                  float* s, void* stream) {
  if (R < 0 || !width_ok(I) || !is16(dtype) || !act_ok(act, limit)) return MOE_ERR_INVALID_ARG;
  const int64_t width = (int64_t)I * (act == MOE_ACT_SRELU ? 1 : 2);
  if (width > INT32_MAX || ldh < width || ldq < width || ldy < I || !maybe(w_row, 4)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  if (R == 0) return MOE_OK;
  if (!have(h, 2) || !have(y, 2) || !q || !have(s, 4)) return MOE_ERR_INVALID_ARG;
  CkptArgs a = {};
  a.h = h; a.ldh = ldh; a.w = w_row; a.R = R; a.I = I; a.dtype = dtype; a.act = ActParams{act, alpha, limit};
  a.y = y; a.ldy = ldy; a.q = q; a.ldq = ldq; a.s = s;
  return done(launch_ckpt_fwd(a, (cudaStream_t)stream));
}

moe_status_t moe_act_ckpt_backward(const void* dy, int64_t lddy, const uint8_t* q, int64_t ldq, const float* s,
                                   const float* w_row, int64_t R, int I, int dtype, int act, float alpha, float limit,
                                   void* dh, int64_t lddh, float* dw_row, void* y, int64_t ldy, void* stream) {
  if (R < 0 || !width_ok(I) || !is16(dtype) || !act_ok(act, limit)) return MOE_ERR_INVALID_ARG;
  const int64_t width = (int64_t)I * (act == MOE_ACT_SRELU ? 1 : 2);
  if (width > INT32_MAX || lddh < width || ldq < width || lddy < I || (y && ldy < I)) return MOE_ERR_INVALID_ARG;
  if (!maybe(w_row, 4) || !maybe(dw_row, 4) || !maybe(y, 2)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  if (R == 0) return MOE_OK;
  if (!have(dy, 2) || !q || !have(s, 4) || !have(dh, 2)) return MOE_ERR_INVALID_ARG;
  CkptArgs a = {};
  a.dy = dy; a.lddy = lddy; a.w = w_row; a.R = R; a.I = I; a.dtype = dtype; a.act = ActParams{act, alpha, limit};
  a.y = y; a.ldy = ldy; a.q = const_cast<uint8_t*>(q); a.ldq = ldq; a.s = const_cast<float*>(s);
  a.dh = dh; a.lddh = lddh; a.dw = dw_row;
  return done(launch_ckpt_bwd(a, (cudaStream_t)stream));
}

moe_status_t moe_fp8_quant_rows(const void* x, int64_t ldx, int64_t R, int C, int dtype, uint8_t* q, int64_t ldq,
                                float* s, int64_t lds, void* stream) {
  if (R < 0 || !width_ok(C) || !is_float(dtype) || ldx < C || ldq < C || lds < blocks_of(C)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  if (R == 0) return MOE_OK;
  if (!have(x, size_of(dtype)) || !q || !have(s, 4)) return MOE_ERR_INVALID_ARG;
  const QuantRowsArgs a = {x, ldx, R, C, dtype, q, ldq, s, lds};
  return done(launch_quant128_rows(a, (cudaStream_t)stream));
}

moe_status_t moe_fp8_quant_weights(const void* w, int64_t w_group, int64_t ldw, int G, int N, int K, int dtype,
                                   uint8_t* q, int64_t q_group, int64_t ldq, float* s, uint8_t* qt, int64_t qt_group,
                                   int64_t ldqt, float* st, void* stream) {
  if (G < 1 || !width_ok(N) || !width_ok(K) || !is_float(dtype) || ldw < K || ldq < K) return MOE_ERR_INVALID_ARG;
  if (G > 1 && (w_group < span(N, K, ldw) || q_group < span(N, K, ldq))) return MOE_ERR_INVALID_ARG;
  if (!have(w, size_of(dtype)) || !q || !have(s, 4)) return MOE_ERR_INVALID_ARG;
  if ((qt != nullptr) != (st != nullptr) || !maybe(st, 4)) return MOE_ERR_INVALID_ARG;
  if (qt && (ldqt < N || (G > 1 && qt_group < span(K, N, ldqt)))) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  const QuantWeightsArgs a = {w, w_group, ldw, G, N, K, dtype, q, q_group, ldq, s, qt, qt_group, ldqt, st};
  return done(launch_quant128_weights(a, (cudaStream_t)stream));
}

moe_status_t moe_mm_workspace_size(int kind, int R, int N, int K, int G, size_t* bytes) {
  if (!bytes || !mm_sizes_ok(R, N, K, G)) return MOE_ERR_INVALID_ARG;
  if (kind != MOE_MM_ROWS && kind != MOE_MM_WGRAD && kind != MOE_MM_FP8) return MOE_ERR_INVALID_ARG;
  *bytes = kStatusBytes + (size_t)mm_part_bytes(kind, R, N, K, G);
  return MOE_OK;
}

moe_status_t moe_grouped_mm(const void* x, int64_t ldx, const void* w, int64_t w_group, int64_t ldw, int trans_w,
                            const int32_t* offsets, int R, int N, int K, int G, int dtype, void* out, int64_t ldo,
                            int out_dtype, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t s = mm_check(MOE_MM_ROWS, R, N, K, G, offsets, ws, ws_bytes);
  if (s != MOE_OK) return s;
  const int wr = trans_w ? K : N, wc = trans_w ? N : K;      // rows and row length of a group's matrix
  if (!is16(dtype) || (out_dtype != dtype && out_dtype != MOE_DT_F32)) return MOE_ERR_INVALID_ARG;
  if ((trans_w != 0 && trans_w != 1) || ldx < K || ldw < wc || ldo < N) return MOE_ERR_INVALID_ARG;
  if (G > 1 && w_group < span(wr, wc, ldw)) return MOE_ERR_INVALID_ARG;
  // rows and groups start on 16 bytes: the tensor copies' rule
  if (!have(w, 16) || ldw % 8 || ldx % 8 || (G > 1 && w_group % 8)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  if (R == 0) return MOE_OK;
  if (!have(x, 16) || !have(out, size_of(out_dtype))) return MOE_ERR_INVALID_ARG;
  MmArgs a = {};
  a.R = R; a.N = N; a.K = K; a.G = G; a.offsets = offsets;
  a.a = x; a.lda = ldx; a.b = w; a.ldb = ldw; a.bg = w_group; a.trans_b = trans_w; a.dtype = dtype;
  a.out = out; a.ldo = ldo; a.out_dtype = out_dtype;
  mm_workspace(a, MOE_MM_ROWS, ws);
  return done(launch_mm16(a, false, (cudaStream_t)stream));
}

moe_status_t moe_grouped_mm_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const int32_t* offsets,
                                  int R, int N, int K, int G, int dtype, void* dw, int64_t dw_group, int64_t lddw,
                                  int out_dtype, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t s = mm_check(MOE_MM_WGRAD, R, N, K, G, offsets, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (!is16(dtype) || (out_dtype != dtype && out_dtype != MOE_DT_F32)) return MOE_ERR_INVALID_ARG;
  if (lddy < N || ldx < K || lddw < K || (G > 1 && dw_group < span(N, K, lddw))) return MOE_ERR_INVALID_ARG;
  if (lddy % 8 || ldx % 8 || !have(dw, size_of(out_dtype))) return MOE_ERR_INVALID_ARG;
  // no rows: the kernel writes zeros and reads neither
  if (R > 0 ? !have(dy, 16) || !have(x, 16) : !maybe(dy, 16) || !maybe(x, 16)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  MmArgs a = {};
  a.R = R; a.N = N; a.K = K; a.G = G; a.offsets = offsets;
  a.a = dy; a.lda = lddy; a.b = x; a.ldb = ldx; a.dtype = dtype;
  a.out = dw; a.ldo = lddw; a.og = dw_group; a.out_dtype = out_dtype;
  mm_workspace(a, MOE_MM_WGRAD, ws);
  return done(launch_mm16(a, true, (cudaStream_t)stream));
}

moe_status_t moe_fp8_mm(const uint8_t* xq, int64_t ldx, const float* xs, int64_t ldxs, const uint8_t* wq,
                        int64_t w_group, int64_t ldw, const float* wscale, const int32_t* offsets, int R, int N, int K,
                        int G, void* out, int64_t ldo, int out_dtype, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t s = mm_check(MOE_MM_FP8, R, N, K, G, offsets, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (!is_float(out_dtype) || ldx < K || ldw < K || ldo < N || ldxs < blocks_of(K)) return MOE_ERR_INVALID_ARG;
  if (G > 1 && w_group < span(N, K, ldw)) return MOE_ERR_INVALID_ARG;
  if (!have(wq, 16) || ldw % 16 || ldx % 16 || (G > 1 && w_group % 16) || !have(wscale, 4)) return MOE_ERR_INVALID_ARG;
  reset_launch_count();
  if (R == 0) return MOE_OK;
  if (!have(xq, 16) || !have(xs, 4) || !have(out, size_of(out_dtype))) return MOE_ERR_INVALID_ARG;
  MmArgs a = {};
  a.R = R; a.N = N; a.K = K; a.G = G; a.offsets = offsets;
  a.a = xq; a.lda = ldx; a.sa = xs; a.ldsa = ldxs; a.b = wq; a.ldb = ldw; a.bg = w_group; a.sb = wscale;
  a.out = out; a.ldo = ldo; a.out_dtype = out_dtype;
  mm_workspace(a, MOE_MM_FP8, ws);
  return done(launch_mm_fp8(a, (cudaStream_t)stream));
}

moe_status_t moe_linear_workspace_size(int R, int rows, int K, int backward, size_t* bytes) {
  if (!bytes || R < 0 || R > kMost || !width_ok(rows) || !width_ok(K) || (backward != 0 && backward != 1))
    return MOE_ERR_INVALID_ARG;
  *bytes = kStatusBytes + (size_t)linear_part_bytes(R, rows, K, backward != 0);
  return MOE_OK;
}

moe_status_t moe_linear_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                                const void* residual, int64_t ldr, int R, int N, int K, int act, float alpha,
                                float limit, int dtype, int wdtype, void* z, int64_t ldz, void* out, int64_t ldo,
                                void* ws, size_t ws_bytes, void* stream) {
  if (!linear_act_ok(act, limit) || !linear_sizes_ok(R, N, K, act)) return MOE_ERR_INVALID_ARG;
  const int rows = act_gated(act) ? 2 * N : N;
  if (!is16(dtype) || (wdtype != MOE_DT_F32 && wdtype != dtype)) return MOE_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldx % 8 || ldw % 8 || ldo < N) return MOE_ERR_INVALID_ARG;
  if ((residual && ldr < N) || (z && ldz < rows) || (residual == out && residual && ldr != ldo)) return MOE_ERR_INVALID_ARG;
  if (!have(w, 16) || !maybe(bias, size_of(wdtype)) || !maybe(residual, 2) || !maybe(z, 2)) return MOE_ERR_INVALID_ARG;
  if (!have(ws, 16)) return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  const moe_status_t s = moe_linear_workspace_size(R, rows, K, 0, &need);
  if (s != MOE_OK) return s;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  reset_launch_count();
  if (R == 0) return MOE_OK;
  if (!have(x, 16) || !have(out, 2)) return MOE_ERR_INVALID_ARG;
  LinearArgs a = {};
  a.R = R; a.N = N; a.K = K; a.act = ActParams{act, alpha, limit}; a.dtype = dtype; a.wdtype = wdtype;
  a.x = x; a.ldx = ldx; a.w = w; a.ldw = ldw; a.bias = bias; a.res = residual; a.ldr = ldr; a.z = z; a.ldz = ldz;
  a.out = out; a.ldo = ldo;
  linear_workspace(a, ws);
  return done(launch_linear_fwd(a, (cudaStream_t)stream));
}

moe_status_t moe_linear_backward(const void* dout, int64_t lddout, const void* x, int64_t ldx, const void* w,
                                 int64_t ldw, const void* z, int64_t ldz, int R, int N, int K, int act, float alpha,
                                 float limit, int dtype, int wdtype, void* dz, int64_t lddz, void* dx, int64_t lddx,
                                 void* dw, int64_t lddw, void* db, void* ws, size_t ws_bytes, void* stream) {
  if (!linear_act_ok(act, limit) || !linear_sizes_ok(R, N, K, act)) return MOE_ERR_INVALID_ARG;
  const int rows = act_gated(act) ? 2 * N : N;
  const bool plain = act == MOE_ACT_NONE;
  if (!is16(dtype) || (wdtype != MOE_DT_F32 && wdtype != dtype)) return MOE_ERR_INVALID_ARG;
  if (lddout < N || ldx < K || ldw < K || ldx % 8 || ldw % 8 || (dx && lddx < K) || (dw && lddw < K))
    return MOE_ERR_INVALID_ARG;
  if (plain ? lddout % 8 != 0 : (ldz < rows || lddz < rows || lddz % 8)) return MOE_ERR_INVALID_ARG;
  if (!maybe(dx, 2) || !maybe(dw, 2) || !maybe(db, size_of(wdtype)) || !maybe(x, 16) || !maybe(w, 16))
    return MOE_ERR_INVALID_ARG;
  if (!have(ws, 16)) return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  const moe_status_t s = moe_linear_workspace_size(R, rows, K, 1, &need);
  if (s != MOE_OK) return s;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  reset_launch_count();
  if (R == 0) {     // the sums over no rows
    const size_t width = (size_t)K * 2;
    if (dw && cudaMemset2DAsync(dw, (size_t)lddw * 2, 0, width, rows, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, rows * size_of(wdtype), st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!have(dout, plain ? 16 : 2) || (!plain && (!have(z, 2) || !have(dz, 16)))) return MOE_ERR_INVALID_ARG;
  if ((dx && !w) || (dw && !x)) return MOE_ERR_INVALID_ARG;
  LinearArgs a = {};
  a.R = R; a.N = N; a.K = K; a.act = ActParams{act, alpha, limit}; a.dtype = dtype; a.wdtype = wdtype;
  a.x = x; a.ldx = ldx; a.w = w; a.ldw = ldw; a.z = const_cast<void*>(z); a.ldz = ldz; a.dout = dout; a.lddout = lddout;
  a.dz = dz; a.lddz = lddz; a.dx = dx; a.lddx = lddx; a.dw = dw; a.lddw = lddw; a.db = db;
  linear_workspace(a, ws);
  return done(launch_linear_bwd(a, st));
}

moe_status_t moe_layer16_workspace_size(int T, int H, int I, int E, int k, int n_shared, size_t* bytes) {
  if (!bytes || !layer16_sizes_ok(T, H, I, E, k, n_shared)) return MOE_ERR_INVALID_ARG;
  if (T > MOE_LAYER16_MAX_T) return MOE_ERR_UNSUPPORTED;
  *bytes = kStatusBytes + (size_t)layer16_ws_bytes(T, H, I, E, k, n_shared);
  return MOE_OK;
}

moe_status_t moe_layer16_forward(const void* x, int64_t ldx, const float* W_r, const float* logits, const void* w1,
                                 int64_t w1_group, int64_t ldw1, const float* b1, const void* w2, int64_t w2_group,
                                 int64_t ldw2, int T, int H, int I, int E, int k, int n_shared, int act, float alpha,
                                 float limit, float routed_scale, int dtype, void* out, int64_t ldo, int32_t* topk_ids,
                                 float* topk_w, void* ws, size_t ws_bytes, void* stream) {
  if (!act_ok(act, limit) || !is16(dtype) || !(routed_scale > 0.f)) return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  const moe_status_t s = moe_layer16_workspace_size(T, H, I, E, k, n_shared, &need);
  if (s != MOE_OK) return s;
  const int rows = act == MOE_ACT_SRELU ? I : 2 * I, G = E + n_shared;
  if ((W_r && logits) || !maybe(W_r, 4) || !maybe(logits, 4) || (b1 && act == MOE_ACT_SRELU) || !maybe(b1, 4))
    return MOE_ERR_INVALID_ARG;
  if (ldx < H || ldw1 < H || ldw2 < I || ldo < H || ldx % 8 || ldw1 % 8 || ldw2 % 8) return MOE_ERR_INVALID_ARG;
  if (G > 1 && (w1_group < span(rows, H, ldw1) || w2_group < span(H, I, ldw2) || w1_group % 8 || w2_group % 8))
    return MOE_ERR_INVALID_ARG;
  if (!have(w1, 16) || !have(w2, 16) || !have(ws, 16)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  reset_launch_count();
  if (T == 0) return MOE_OK;
  if (!have(x, 16) || !have(out, 2) || !have(topk_ids, 4) || !have(topk_w, 4)) return MOE_ERR_INVALID_ARG;
  Layer16Args a = {};
  a.T = T; a.H = H; a.I = I; a.E = E; a.k = k; a.S = n_shared; a.act = ActParams{act, alpha, limit}; a.rs = routed_scale;
  a.dtype = dtype; a.x = x; a.ldx = ldx; a.W_r = W_r; a.logits = logits; a.w1 = w1; a.g1 = w1_group; a.ld1 = ldw1;
  a.b1 = b1; a.w2 = w2; a.g2 = w2_group; a.ld2 = ldw2; a.out = out; a.ldo = ldo; a.ids = topk_ids; a.w = topk_w;
  a.status = reinterpret_cast<int32_t*>(ws); a.ws = reinterpret_cast<uint8_t*>(ws) + kStatusBytes;
  a.arrive = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(ws) + kArriveAt);
  return done(launch_layer16(a, (cudaStream_t)stream));
}

moe_status_t moe_mm_read_status(void* ws, int32_t* out, void* stream) {
  if (!have(ws, 16) || !out) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(out, ws, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemsetAsync(ws, 0, 4, st) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_ERR_CUDA;
  return *out ? MOE_ERR_DEVICE : MOE_OK;
}

}  // extern "C"
