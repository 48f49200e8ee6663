// The norms' backward pass from an e4m3 checkpoint and 16-bit dy (norm_ring.cuh); a file of its own, as files compile in parallel.
#include "norm_ring.cuh"

namespace rlk {

cudaError_t launch_norm_rows_e4m3_bf16(const NormBackwardParams &p, const NormTeams &n, int blocks, cudaStream_t stream) {
    return launch_norm_rows<kHE4M3, true>(p, n, blocks, stream);
}

}  // namespace rlk
