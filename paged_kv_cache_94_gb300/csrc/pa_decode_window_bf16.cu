// Compiled decode kernels over a window and the sequence's first tokens (PASS 1):
// bf16 K/V, head dims 64 and 128, group sizes 1..16. Warps, ring stages and blocks
// per item are the plain decode's.
//
//     out[b][h] = sum_j softmax(scale <q[b][h], K_b[j]>)_j V_b[j] over j < ctx_b with
//     j >= ctx_b - window or j < n_first
//
// Bound by HBM: n_first + window rows of K and V per (sequence, kv head), whose blocks lie on
// the line without those between the two (kept_blocks, skipped_blocks), so that a window takes
// what a context of its length takes, wherever it begins. Measured on a GB300: 64 sequences of
// 512..16384 tokens, 32 / 8 heads of 128, a window of 4096 and 4 first tokens: 146 us, 6600
// GB/s, 0.97 of the measured copy rate; one sequence, a window of 1024: 9.4 us (latency).
#include "pa_decode_kernel.cuh"

namespace pa {
namespace {

template <int D, int G>
struct PolOf;
template <int G>
struct PolOf<128, G> {
    using type = Bf16Policy<128, G, (G >= 16 ? 4 : 8), 2>;
};
template <int G>
struct PolOf<64, G> {
    using type = Bf16Policy<64, G, 4, 6>;
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

const DecodeKernel *find_window_kernel_bf16(int d_h, int group)
{
    return d_h == 128 ? find<128>(group) : d_h == 64 ? find<64>(group) : nullptr;
}

} // namespace pa
