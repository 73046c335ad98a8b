// Rotary positions with the append: queries and keys are turned by their positions, keys and
// values go to the paged pool, in one pass.
//
// Pair i < pairs of a head turns by angle_i = positions[axis_i][t] * inv_freq[i]:
//     (a, b) -> amplitude (a cos - b sin, b cos + a sin)
// where (a, b) are values (i, i + pairs) or (2 i, 2 i + 1); values from 2 * pairs on stay.
//
// Angles. In 32 bits position * inv_freq of a far position has lost the angle (2^20 rad: steps
// of 1/16). Here a frequency is a 64-bit fraction of a turn, and its product with the position
// modulo 2^64 drops whole turns exactly. What is left, less whole quarters, is rounded once to
// fp32 (an angle below pi / 4, 2^-24 relative).
//
// What bounds it: memory for prompts (each row read once and written once), latency for a
// decode step. A thread takes 16 values of a row, both halves of its eight pairs, as two
// 16-byte pieces; a CTA some tokens, whose sines and cosines it works out once for all heads
// while the first rows are on their way.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;
constexpr int kMaxTokens = 32; // of one CTA

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride; // elements from token to token
    __nv_bfloat16 *out;
    const int32_t *positions; // [n_axes][num_tokens]
    const double *inv_freq;
    const int32_t *axis; // NULL: all on axis 0
    const int64_t *slots;
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int32_t *dev_status;
    int64_t num_tokens, num_slots;
    float amplitude;
    int32_t n_axes, pairs, n_h, n_kv;
    int32_t tokens; // of one CTA
    int32_t rows;   // of a token: n_h + 2 n_kv
    int32_t adjacent;
};

// cos and sin of position * freq, freq in radians per position.
__device__ __forceinline__ float2 turn_of(int32_t position, double freq, float amplitude)
{
    const double turns = freq * 0.15915494309189533577; // 1 / (2 pi)
    if (!(fabs(turns) < 4.5e15)) // no fraction left, or not a number
        return make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
    const int64_t step = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
    const uint64_t at = (uint64_t)(int64_t)position * (uint64_t)step;
    const uint64_t quarter = (at + (1ull << 61)) >> 62; // nearest
    // half turns, -1/4 .. 1/4
    const float x = (float)(int64_t)(at - (quarter << 62)) * 1.0842021724855044e-19f; // 2^-63
    float s, c;
    sincospif(x, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    if (quarter & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c * amplitude, s * amplitude);
}

__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8])
{
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Codes of eight values (the quantiser of pa_cache_write).
template <int KIND>
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float scale)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float c = 0.f;
        if (scale != 0.f) {
            c = rintf(__fdiv_rn(x[i], scale));
            c = KIND == 1 ? fminf(fmaxf(c, -128.f), 127.f) : fminf(fmaxf(c, -8.f), 7.f);
        }
        if constexpr (KIND == 1)
            w[i / 4] |= (uint32_t)(uint8_t)(int8_t)(int)c << (8 * (i % 4));
        else
            w[0] |= ((uint32_t)(int)c & 0xFu) << (4 * i);
    }
    return make_uint2(w[0], w[1]);
}

// KIND: 0 bf16, 1 INT8, 2 INT4; U: pieces of a thread whose loads are in flight together
template <int D, int KIND, int U>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const RopeParams p)
{
    // a decode launched next on the stream may be scheduled now; it waits for
    // this grid to complete before reading the cache
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int PPR = D / 16; // pieces of a row
    __shared__ float2 turns[kMaxTokens * kMaxPairs];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, p.num_tokens - t0);
    const int per_token = p.rows * PPR, pieces = tokens * per_token;
    bool made = false;
    for (int i0 = blockIdx.y * (kThreads * U) + tid; i0 - tid < pieces;
         i0 += gridDim.y * (kThreads * U)) {
        uint4 a[U], b[U];
        int tok[U], row[U], from[U], step[U]; // a piece's values: from .. + 7, from + step ..
        int64_t slot[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            live[u] = i < pieces;
            tok[u] = live[u] ? i / per_token : 0;
            const int r = live[u] ? i - tok[u] * per_token : 0, c = r % PPR;
            row[u] = r / PPR;
            const bool halves = !p.adjacent && 8 * c < p.pairs;
            from[u] = halves ? 8 * c : 16 * c;
            step[u] = halves ? p.pairs : 8;
            const int h = row[u];
            const int64_t t = t0 + tok[u];
            const __nv_bfloat16 *src =
                h < p.n_h            ? p.q + t * p.q_stride + h * D
                : h < p.n_h + p.n_kv ? p.k + t * p.k_stride + (h - p.n_h) * D
                                     : p.v + t * p.v_stride + (h - p.n_h - p.n_kv) * D;
            a[u] = b[u] = make_uint4(0, 0, 0, 0);
            slot[u] = live[u] && h >= p.n_h ? p.slots[t] : -1;
            if (live[u]) {
                a[u] = *reinterpret_cast<const uint4 *>(src + from[u]);
                b[u] = *reinterpret_cast<const uint4 *>(src + from[u] + step[u]);
            }
        }
        if (!made) {
            made = true;
            for (int j = tid; j < tokens * p.pairs; j += kThreads) {
                const int t = j / p.pairs, i = j - t * p.pairs;
                const int axis = p.axis ? p.axis[i] : 0;
                float2 cs = make_float2(1.f, 0.f); // (an axis that is not there turns nothing)
                if (axis >= 0 && axis < p.n_axes)
                    cs = turn_of(p.positions[axis * p.num_tokens + t0 + t], p.inv_freq[i],
                                 p.amplitude);
                else if (p.dev_status)
                    atomicOr(p.dev_status, PA_DEV_BAD_CONTEXT_BIT);
                turns[t * kMaxPairs + i] = cs;
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[8], y[8];
            unpack(a[u], x);
            unpack(b[u], y);
            const bool is_v = row[u] >= p.n_h + p.n_kv;
            const int pair = p.adjacent ? from[u] / 2 : from[u];
            if (!is_v && (p.adjacent ? from[u] < 2 * p.pairs
                                     : step[u] == p.pairs && from[u] < p.pairs)) {
                const float4 *cs =
                    reinterpret_cast<const float4 *>(turns + tok[u] * kMaxPairs + pair);
#pragma unroll
                for (int e = 0; e < 4; ++e) { // two pairs at a time
                    const float4 w = cs[e];
                    if (p.adjacent) {
                        float *z = e < 2 ? x + 4 * e : y + 4 * (e - 2);
                        const float a0 = z[0], b0 = z[1], a1 = z[2], b1 = z[3];
                        z[0] = a0 * w.x - b0 * w.y;
                        z[1] = b0 * w.x + a0 * w.y;
                        z[2] = a1 * w.z - b1 * w.w;
                        z[3] = b1 * w.z + a1 * w.w;
                    } else {
                        const float a0 = x[2 * e], b0 = y[2 * e], a1 = x[2 * e + 1],
                                    b1 = y[2 * e + 1];
                        x[2 * e] = a0 * w.x - b0 * w.y;
                        y[2 * e] = b0 * w.x + a0 * w.y;
                        x[2 * e + 1] = a1 * w.z - b1 * w.w;
                        y[2 * e + 1] = b1 * w.z + a1 * w.w;
                    }
                }
            }
            const int64_t t = t0 + tok[u];
            if (row[u] < p.n_h && live[u]) {
                __nv_bfloat16 *dst = p.out + (t * p.n_h + row[u]) * D + from[u];
                *reinterpret_cast<uint4 *>(dst) = pack(x);
                *reinterpret_cast<uint4 *>(dst + step[u]) = pack(y);
            }
            float scale = 0.f;
            if constexpr (KIND != 0) { // (all lanes of a warp take part)
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
                for (int o = PPR / 2; o > 0; o >>= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale = __fdiv_rn(m, KIND == 1 ? 127.f : 7.f);
            }
            if (row[u] < p.n_h || !live[u])
                continue;
            const int64_t s = slot[u];
            const int h = row[u] - p.n_h - (is_v ? p.n_kv : 0);
            const bool lead = from[u] == 0;
            if (s < 0 || s >= p.num_slots) {
                if (s >= 0 && lead && h == 0 && p.dev_status)
                    atomicOr(p.dev_status, PA_DEV_BAD_SLOT_BIT);
                continue;
            }
            const int64_t dst_row = ((s >> 4) * p.n_kv + h) * 16 + (s & 15);
            void *pool = is_v ? p.v_cache : p.k_cache;
            if constexpr (KIND == 0) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(pool) + dst_row * D + from[u];
                *reinterpret_cast<uint4 *>(dst) = is_v ? a[u] : pack(x);
                *reinterpret_cast<uint4 *>(dst + step[u]) = is_v ? b[u] : pack(y);
            } else {
                const uint2 cx = codes_of<KIND>(x, scale), cy = codes_of<KIND>(y, scale);
                if constexpr (KIND == 1) {
                    int8_t *dst = static_cast<int8_t *>(pool) + dst_row * D + from[u];
                    *reinterpret_cast<uint2 *>(dst) = cx;
                    *reinterpret_cast<uint2 *>(dst + step[u]) = cy;
                } else {
                    uint8_t *dst = static_cast<uint8_t *>(pool) + (dst_row * D + from[u]) / 2;
                    *reinterpret_cast<uint32_t *>(dst) = cx.x;
                    *reinterpret_cast<uint32_t *>(dst + step[u] / 2) = cy.x;
                }
                if (lead)
                    (is_v ? p.v_scale : p.k_scale)[dst_row] = scale;
            }
        }
    }
}

template <int D, int KIND>
cudaError_t launch_of(const RopeParams &p, int sms, cudaStream_t stream)
{
    using std::max;
    using std::min;
    RopeParams r = p;
    const int per_token = p.rows * (D / 16);
    const int64_t all = p.num_tokens * per_token;
    const int64_t few = (int64_t)sms * 2 * kThreads; // pieces that go one to a thread
    if (all <= few) {
        r.tokens = 1;
        const dim3 grid((unsigned)p.num_tokens, (unsigned)((per_token + kThreads - 1) / kThreads));
        rope_write_kernel<D, KIND, 1><<<grid, kThreads, 0, stream>>>(r);
    } else {
        r.tokens = max(1, min(kMaxTokens, 4 * kThreads / per_token));
        const int64_t blocks = (p.num_tokens + r.tokens - 1) / r.tokens;
        if (blocks > 0x7fffffff)
            return cudaErrorInvalidValue;
        rope_write_kernel<D, KIND, 4><<<(unsigned)blocks, kThreads, 0, stream>>>(r);
    }
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_rope_write(const RopeArgs &a, int sms, cudaStream_t stream)
{
    RopeParams p;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.axis = a.axis;
    p.slots = a.slots;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.dev_status = a.dev_status;
    p.num_tokens = a.num_tokens;
    p.num_slots = a.num_blocks * 16;
    p.amplitude = a.amplitude;
    p.n_axes = a.n_axes;
    p.pairs = a.pairs;
    p.n_h = a.n_h;
    p.n_kv = a.n_kv;
    p.tokens = 1;
    p.rows = a.n_h + 2 * a.n_kv;
    p.adjacent = a.adjacent;
    if (a.d_h == 128)
        return a.kind == 0   ? launch_of<128, 0>(p, sms, stream)
               : a.kind == 1 ? launch_of<128, 1>(p, sms, stream)
                             : launch_of<128, 2>(p, sms, stream);
    return a.kind == 0   ? launch_of<64, 0>(p, sms, stream)
           : a.kind == 1 ? launch_of<64, 1>(p, sms, stream)
                         : launch_of<64, 2>(p, sms, stream);
}

} // namespace pa
