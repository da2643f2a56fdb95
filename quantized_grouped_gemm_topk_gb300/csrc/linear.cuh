// What the dense products share: linear.cu (entries, backward's dz) and the kernel of
// many rows (linear_pairs.cuh), one source for each type.
#pragma once
#include "few16.cuh"

namespace moe {

// D[M][N] of a tile: out = x w^T | dx = dz w | dw = dz^T x.
enum { kLinFwd = 0, kLinDx = 1, kLinDw = 2 };
struct LinArgs {
  LinearArgs a;
  int64_t M;            // rows of the result,
  int N, K;             // its columns (gated: of out), the reduction
  uint16_t* out; int64_t ldo;
  int bn;               // columns of an MMA: the tile's, gated twice those
  int mt, nt;           // tiles of rows and of columns
  int group;            // tiles of rows that follow each other before the next column tile
};

__host__ __device__ __forceinline__ bool rows16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

// The product of g on pairs of SMs.
cudaError_t launch_pairs_bf16(LinArgs& g, int mode, bool gated, cudaStream_t st);
cudaError_t launch_pairs_f16(LinArgs& g, int mode, bool gated, cudaStream_t st);

}  // namespace moe
