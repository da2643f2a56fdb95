// The dense products of many rows, f16.
#include "linear_pairs.cuh"

namespace moe {

cudaError_t launch_pairs_f16(LinArgs& g, int mode, bool gated, cudaStream_t st) { return launch_pairs<F16>(g, mode, gated, st); }

}  // namespace moe
