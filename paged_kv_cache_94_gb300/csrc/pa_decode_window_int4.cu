// Compiled decode kernels over a window and the sequence's first tokens (PASS 1):
// int4 K/V, head dims 64 and 128, group sizes 1..16. Warps, ring stages and blocks
// per item are the plain decode's. 96 sequences of 1..3001 tokens, 16 heads of 64,
// g = 1, a window of 1001 and 20 first tokens: 54 us on a GB300, 1730 GB/s, 0.26 of the measured
// copy rate; bound by its instructions (one of the contraction's eight columns is live) and their
// latency: with 11 warps per SM the issue slots are 50% busy, most of the rest fixed latencies
// between dependent instructions. 61 with values that all take weights in two parts.
#include "pa_decode_kernel.cuh"

namespace pa {
namespace {

template <int D, int G>
struct PolOf;
template <int G>
struct PolOf<128, G> {
    using type = QuantMmaPolicy<4, 128, G, 4, 2, (G >= 16 ? 1 : 3), 2, 1, false>;
};
template <int G>
struct PolOf<64, G> {
    using type = QuantMmaPolicy<4, 64, G, 4, 4, (G > 8 ? 1 : 3), 2, 1, false>;
};

template <int D, int G>
using Pol = typename PolOf<D, G>::type;

template <class P>
size_t smem_of(int num_seqs)
{
    return P::Layout::bytes(num_seqs);
}

template <class P>
cudaError_t launch_of(const CUtensorMap &tk, const CUtensorMap &tv, const DecodeParams &p, int grid,
                      size_t smem, cudaStream_t stream)
{
    return launch_decode<P, 1>(tk, tv, p, grid, smem, stream);
}

template <int D, int G>
const DecodeKernel kEntry = {reinterpret_cast<const void *>(&decode_kernel<Pol<D, G>, 1>),
                             Pol<D, G>::NW * 32, &smem_of<Pol<D, G>>, &launch_of<Pol<D, G>>};

template <int D>
const DecodeKernel *find(int group)
{
    switch (group) {
    case 1: return &kEntry<D, 1>;
    case 2: return &kEntry<D, 2>;
    case 4: return &kEntry<D, 4>;
    case 8: return &kEntry<D, 8>;
    case 16: return &kEntry<D, 16>;
    default: return nullptr;
    }
}

} // namespace

const DecodeKernel *find_window_kernel_int4(int d_h, int group)
{
    return d_h == 128 ? find<128>(group) : d_h == 64 ? find<64>(group) : nullptr;
}

} // namespace pa
