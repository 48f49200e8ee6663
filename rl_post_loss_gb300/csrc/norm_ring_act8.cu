// The norms' backward pass from an 8-bit checkpoint (norm_ring.cuh); a file of its own, as the build compiles files in parallel.
#include "norm_ring.cuh"

namespace rlk {

cudaError_t launch_norm_ring_act8(const NormBackwardParams &p, const NormRing &r, int parts, cudaStream_t stream) {
    if (p.dx.bf16) return launch_norm_ring_shape<kHAct8, true, true>(p, r, parts, stream);
    return p.dy.bf16 ? launch_norm_ring_shape<kHAct8, false, true>(p, r, parts, stream) : launch_norm_ring_shape<kHAct8, false, false>(p, r, parts, stream);
}

}  // namespace rlk
