// Compiled cross-attention kernels (pa_cross_kernel.cuh without its mask).
#include "pa_cross_kernel.cuh"

namespace pa {

size_t cross_workspace_bytes(int d_h, int num_ctas)
{
    return counter_bytes(num_ctas) + (size_t)num_ctas * 2 * record_floats(d_h) * sizeof(float);
}

cudaError_t launch_cross(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                         const CrossArgs &a, cudaStream_t stream)
{
    return launch_any<0>(tq, tk, tv, a, stream);
}

} // namespace pa
