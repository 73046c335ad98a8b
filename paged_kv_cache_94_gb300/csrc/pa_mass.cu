// Attention weights of a decode step, added to each cached token's mass.
//
// The decode kernel (MASS instance) leaves the scores s (log2 domain) of every
// attended token, [b][kv head][token][g], and each query row's softmax base M
// and reciprocal sum 1/L. With those,
//     w[b][kvh][j] = sum_h 2^(s_jh - M_h) / L_h,   mass_out = mass + w,
// one pass over the scores: g fp32 read per token and kv head, 4 bytes of mass
// read and 4 written, no atomics, so the sums do not depend on any order. Keeping
// the scores costs 8 g bytes a token against the 4 d_h (bf16) of its K and V
// rows; working them out a second time would read the K half again.
//
// HBM- or L2-bound: 9 us on top of the decode's 96 for 64 sequences of 512..4096 tokens
// (bf16, 32 heads on 8), 14 on 122 for four of 32K..128K (INT8). Each thread takes four adjacent tokens, so masses move as
// float4 whatever g is; units (b, kv head) are cut over blockIdx.y so that few
// long contexts still fill the GPU.
#include "pa_decode.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

template <int G>
__global__ void __launch_bounds__(kThreads)
mass_kernel(const float *__restrict__ scores, const float2 *__restrict__ ml,
            const int32_t *__restrict__ context_lens, const float *mass, float *mass_out, int n_kv,
            int max_blocks)
{
    // (programmatic dependent launch: the decode's results are complete after this)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t u = blockIdx.x; // b * n_kv + kv head
    const int32_t ctx = __ldg(context_lens + u / n_kv);
    const int64_t cap = (int64_t)max_blocks * kBlockTokens;
    if (ctx <= 0 || ctx > cap)
        return; // nothing attended (a bad length was reported by the decode)
    float M[G], R[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
        const float2 v = __ldcg(ml + u * G + h);
        // every score of the row -inf: no weight anywhere
        M[h] = v.x == -INFINITY ? 0.f : v.x;
        R[h] = v.x == -INFINITY ? 0.f : v.y;
    }
    const float4 *sc = reinterpret_cast<const float4 *>(scores + u * cap * G);
    for (int64_t t = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * 4; t < ctx;
         t += (int64_t)gridDim.y * kThreads * 4) {
        float s[4 * G];
#pragma unroll
        for (int i = 0; i < G; ++i) { // the 4 tokens' scores: G float4 (cap * G is a multiple of 4)
            const float4 v = __ldcs(sc + t / 4 * G + i);
            s[4 * i] = v.x;
            s[4 * i + 1] = v.y;
            s[4 * i + 2] = v.z;
            s[4 * i + 3] = v.w;
        }
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h)
                w[j] = fmaf(fast_exp2(s[j * G + h] - M[h]), R[h], w[j]);
        }
        const int64_t at = u * cap + t;
        if (t + 4 <= ctx) {
            const float4 m = *reinterpret_cast<const float4 *>(mass + at);
            *reinterpret_cast<float4 *>(mass_out + at) =
                make_float4(m.x + w[0], m.y + w[1], m.z + w[2], m.w + w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (t + j < ctx)
                    mass_out[at + j] = mass[at + j] + w[j];
        }
    }
}

} // namespace

cudaError_t launch_mass(const float *scores, const float2 *ml, const int32_t *context_lens,
                        const float *mass, float *mass_out, int num_seqs, int n_kv, int g,
                        int max_blocks, int sms, cudaStream_t stream)
{
    const int64_t units = (int64_t)num_seqs * n_kv;
    const int64_t rounds = ((int64_t)max_blocks * kBlockTokens + 4 * kThreads - 1) / (4 * kThreads);
    // about eight CTAs per SM, but no more per unit than the longest context could use
    int64_t y = (8 * (int64_t)sms + units - 1) / units;
    y = y < rounds ? y : rounds;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units, (unsigned)y);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, scores, ml, context_lens, mass, mass_out, n_kv,
                                  max_blocks);
    };
    switch (g) {
    case 1: return go(mass_kernel<1>);
    case 2: return go(mass_kernel<2>);
    case 4: return go(mass_kernel<4>);
    case 8: return go(mass_kernel<8>);
    case 16: return go(mass_kernel<16>);
    default: return cudaErrorInvalidValue;
    }
}

const DecodeKernel *find_mass_kernel_bf16(int d_h, int group);
const DecodeKernel *find_mass_kernel_int8(int d_h, int group);
const DecodeKernel *find_mass_kernel_int4(int d_h, int group);

const DecodeKernel *find_mass_kernel(int kind, int d_h, int group)
{
    return kind == 0   ? find_mass_kernel_bf16(d_h, group)
           : kind == 1 ? find_mass_kernel_int8(d_h, group)
           : kind == 2 ? find_mass_kernel_int4(d_h, group)
                       : nullptr;
}

} // namespace pa
