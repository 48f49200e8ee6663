// The norms' backward pass from 32-bit rows and 32-bit dy (norm_ring.cuh); a file of its own, as files compile in parallel.
#include "norm_ring.cuh"

namespace rlk {

cudaError_t launch_norm_rows_f32_f32(const NormBackwardParams &p, const NormTeams &n, int blocks, cudaStream_t stream) {
    return launch_norm_rows<kHF32, false>(p, n, blocks, stream);
}

}  // namespace rlk
