// The forward pass of the norms on rows that start anywhere (norm_fwd.cuh); a file of its own, as files compile in parallel.
#include "norm_fwd.cuh"

namespace rlk {

cudaError_t launch_norm_forward_any(const NormForwardParams &p, const NormTeams &n, cudaStream_t stream) {
    if (p.x.bf16) return n.vecs == 1 ? launch_forward_rows<true, 1, true, kAnyRow>(p, n, stream) : launch_forward_rows<true, 2, true, kAnyRow>(p, n, stream);
    return n.vecs == 1 ? launch_forward_rows<false, 1, true, kAnyRow>(p, n, stream) : launch_forward_rows<false, 2, true, kAnyRow>(p, n, stream);
}
cudaError_t launch_norm_forward_shift(const NormForwardParams &p, const NormTeams &n, cudaStream_t stream) {
    return p.x.bf16 ? launch_forward_vecs<true, true, kShiftRow>(p, n, stream) : launch_forward_vecs<false, true, kShiftRow>(p, n, stream);
}

}  // namespace rlk
