// The norms' backward pass from an int8 checkpoint and 32-bit dy (norm_ring.cuh); a file of its own, as files compile in parallel.
#include "norm_ring.cuh"

namespace rlk {

cudaError_t launch_norm_rows_int8_f32(const NormBackwardParams &p, const NormTeams &n, int blocks, cudaStream_t stream) {
    return launch_norm_rows<kHInt8, false>(p, n, blocks, stream);
}

}  // namespace rlk
