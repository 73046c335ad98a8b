// Compiled kernels of causal attention within a sliding window and to a sequence's first
// tokens (pa_cross_kernel.cuh with its mask).
#include "pa_cross_kernel.cuh"

namespace pa {

cudaError_t launch_window(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const CrossArgs &a, cudaStream_t stream)
{
    return launch_any<true>(tq, tk, tv, a, stream);
}

} // namespace pa
