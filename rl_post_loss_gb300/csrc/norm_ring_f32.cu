// The norms' backward pass from 32-bit rows (norm_ring.cuh); a file of its own, as the build compiles files in parallel.
#include "norm_ring.cuh"

namespace rlk {

cudaError_t launch_norm_ring_f32(const NormBackwardParams &p, const NormRing &r, int parts, cudaStream_t stream) {
    return p.dy.bf16 ? launch_norm_ring_shape<kHF32, false, true>(p, r, parts, stream) : launch_norm_ring_shape<kHF32, false, false>(p, r, parts, stream);
}

}  // namespace rlk
