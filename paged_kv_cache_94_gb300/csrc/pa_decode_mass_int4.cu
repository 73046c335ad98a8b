// Compiled decode kernels that keep their scores (see pa_mass.cu): int4 K/V,
// head dims 64 and 128, group sizes 1..16. Warps, ring stages and blocks per
// item are the plain decode's.
#include "pa_decode_kernel.cuh"

namespace pa {
namespace {

template <int D, int G>
struct PolOf;
template <int G>
struct PolOf<128, G> {
    using type = QuantMmaPolicy<4, 128, G, 4, 2, (G >= 16 ? 1 : 3), 2, 1, false>;
};
// Three resident CTAs per SM, as the plain decode's registers allow up to this g without being
// told (the score stores take a few more: left alone, 170 to 175 against its 168).
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
    return launch_decode<P, 0, true>(tk, tv, p, grid, smem, stream);
}

template <int D, int G>
const DecodeKernel kEntry = {reinterpret_cast<const void *>(&decode_kernel<Pol<D, G>, 0, true>),
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

const DecodeKernel *find_mass_kernel_int4(int d_h, int group)
{
    return d_h == 128 ? find<128>(group) : d_h == 64 ? find<64>(group) : nullptr;
}

} // namespace pa
