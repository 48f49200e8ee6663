// The norms' backward pass from 16-bit rows (norm_ring.cuh); a file of its own, as the build compiles files in parallel.
#include "norm_ring.cuh"

namespace rlk {

cudaError_t launch_norm_ring_bf16(const NormBackwardParams &p, const NormRing &r, int parts, cudaStream_t stream) {
    return launch_norm_ring_shape<kHBf16, true, true>(p, r, parts, stream);
}

}  // namespace rlk
