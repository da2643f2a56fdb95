// Products of 16-bit weights with a few rows (few16.cu): what the layer for a few
// tokens and the dense product hand over.
#pragma once
#include "ops.cuh"

namespace moe {

// Most rows of the dense product here, and most CTAs of the layer (for which the
// workspace has places).
constexpr int kFewRows = 256;
constexpr int kFewSms = 152;

inline int64_t up(int64_t n, int64_t t) { return (n + t - 1) / t; }      // n / t, rounded up

struct FewArgs {
  int R;                      // rows; layer: tokens (at most 64)
  int K1, F1;                 // first product: reduction, features (gated: of a half)
  int K2, F2;                 // layer: second product
  ActParams act;
  int dtype, wdtype;
  int32_t* status;
  // layer
  int E, k, S;
  const int32_t* ids; const float* wts;   // [R][k]
  const float* b1;            // nullable, [E + S][2 F1]
  uint16_t* y; int64_t ldy;   // rows of the second product, by group; of their second part the same behind all of them
  int32_t* ticket;            // zero on entry: ranges claimed,
  int32_t* done;              // ranges of the first product done,
  int32_t* joined;            // [kFewSms] parts of a range of the second done
  float* part;                // [kFewSms][R][128] their sums
  // dense
  const void* bias; const void* res; int64_t ldr; void* z; int64_t ldz;
  void* out; int64_t ldo;     // both
  // set by the launch
  int N;                      // of the MMA; dense: rows a tile
  int rows1;                  // most features a tile
  int head, stages;           // bytes in front of the ring, its stages
  int nt, mt1;                // dense: tiles of rows and of features
  int hs, lanes;              // dense: 64s of the reduction a stage, features side by side in the epilogue
  int issuers;                // warps that issue MMAs; `stages` is a multiple of them
  int ncol;                   // layer: columns of an accumulator
  int Pf, S2;                 // layer: ranges of the second product's features, parts of the groups for each
  int xrows, box2;            // layer: rows of x a copy takes, features of the second product's tiles
  int slot;                   // bytes of a stage
  int hs1[8], ns1[8], hs2[4], ns2[4];   // layer: 64s of the reduction a stage and stages, by the tile's copies
};
cudaError_t launch_few_layer(FewArgs g, const void* x, int64_t ldx, const void* w1, int64_t g1, int64_t ld1, const void* w2,
                             int64_t g2, int64_t ld2, cudaStream_t st);
cudaError_t launch_few_linear(FewArgs g, const void* x, int64_t ldx, const void* w, int64_t ldw, cudaStream_t st);

}  // namespace moe
