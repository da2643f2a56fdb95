// Products of 16-bit weights with a few rows (few16.cu): what the layer for a few
// tokens and the dense product hand over.
#pragma once
#include "ops.cuh"

namespace moe {

// Most rows of the dense product, and most shares (CTAs) the layer's products are cut into.
constexpr int kFewRows = 256;
constexpr int kFewShares = 152;

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
  uint16_t* y; int64_t ldy;   // rows of the second product, by group
  float* zrow; int64_t ldz32; // its results, fp32, by row
  int32_t* ticket;            // zero on entry: shares claimed,
  int32_t* done;              // tiles of the first product,
  int32_t* split2;            // [mt2] shares done with a feature tile
  float* part;                // partial sums: 2 kFewShares slots of N x 128 fp32
  int32_t* split;             // [kFewShares] pieces done of the tiles that span shares; zero on entry
  // dense
  const void* bias; const void* res; int64_t ldr; void* z; int64_t ldz;
  void* out; int64_t ldo;     // both
  // set by the launch
  int N, nt, rows1, mt1, nk1, mt2, nk2, least, head, stages;    // nt: dense, tiles of N rows
};
cudaError_t launch_few_layer(FewArgs g, const void* x, int64_t ldx, const void* w1, int64_t g1, int64_t ld1, const void* w2,
                             int64_t g2, int64_t ld2, cudaStream_t st);
cudaError_t launch_few_linear(FewArgs g, const void* x, int64_t ldx, const void* w, int64_t ldw, cudaStream_t st);
// Bytes of the layer's partial sums for R tokens.
inline int64_t few_part_bytes(int R) { return (int64_t)2 * kFewShares * ((R + 15) & ~15) * 128 * 4; }

}  // namespace moe
