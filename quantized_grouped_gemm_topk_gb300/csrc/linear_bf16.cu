// The dense products of many rows, bf16.
#include "linear_pairs.cuh"

namespace moe {

cudaError_t launch_pairs_bf16(LinArgs& g, int mode, bool gated, cudaStream_t st) { return launch_pairs<Bf16>(g, mode, gated, st); }

}  // namespace moe
