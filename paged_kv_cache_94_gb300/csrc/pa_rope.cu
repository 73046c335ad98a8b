// Rotary positions with the append: queries and keys are turned by their positions, keys and
// values go to the paged pool, in one pass.
//
// Pair i < pairs of a head turns by angle_i = positions[axis_i][t] * inv_freq[i]:
//     (a, b) -> amplitude (a cos - b sin, b cos + a sin)
// where (a, b) are values (i, i + pairs) or (2 i, 2 i + 1); values from 2 * pairs on stay.
//
// Angles. In 32 bits position * inv_freq of a far position has lost the angle (2^20 rad: steps
// of 1/16). Here a frequency is a 64-bit fraction of a turn, and its product with the position
// modulo 2^64 drops whole turns exactly. What is left, less whole quarters, is an angle of up to
// pi / 4 in fp32, whose sine and cosine need a few products.
//
// What bounds it: memory for prompts (each row read once and written once), latency for a
// decode step. A thread takes 16 values of a row, both halves of its eight pairs, as two
// 16-byte loads, the same ones of every row that it comes to; a CTA some tokens, whose sines
// and cosines it works out once for all heads while the first rows are on their way.
//
// Measured on a GB300, launches back to back: 8192 tokens of 32 + 8 heads of 128 into a bf16
// pool 37.7 us, 5340 GB/s, 0.79 of the measured copy rate (56 with rows found by division and
// 98 registers, two CTAs per SM; 39 with angles in double precision); into an INT8 pool 42.
// 4111 tokens of 16 + 16 heads of 64 into an INT8 pool 12.8 us, INT4 12.5, bf16 8.6 (INT8 21.5
// where one near half had all eight values divided, 18.7 with a division each); issue slots 62%
// busy, most of a warp's time ready and not picked. A step of 64 tokens 2.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

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
    int32_t rows;   // of a token: n_h + 2 n_kv
    int32_t tokens; // of one CTA
    int32_t round_rows, round_tokens; // how far a thread's row moves from round to round
};

// freq (radians per position) in turns, times 2^64 and modulo 2^64. In integers: a CTA's few
// multiplications in double precision would keep that unit, a 64th as fast, busy for 800 cycles.
// freq = m 2^(e - 52), 1 / (2 pi) = c 2^-64 within 2^-62 of itself: m c 2^(e - 52).
__device__ __forceinline__ uint64_t turn_step(double freq)
{
    const uint64_t bits = (uint64_t)__double_as_longlong(freq);
    const int e = (int)(bits >> 52 & 0x7ff) - 1023;
    const uint64_t m = (bits & 0xfffffffffffffull) | 1ull << 52, c = 0x28be60db9391054aull;
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    const int right = 52 - e; // how far the product moves
    uint64_t x;
    if (right >= 128 || right <= -64)
        x = 0;
    else if (right >= 64)
        x = hi >> (right - 64);
    else if (right > 0)
        x = lo >> right | hi << (64 - right);
    else
        x = lo << -right;
    return (bits >> 63) ? 0 - x : x;
}

// cos and sin of position * freq.
__device__ __forceinline__ float2 turn_of(int32_t position, double freq, float amplitude)
{
    if ((__double2hiint(freq) & 0x7ff00000) == 0x7ff00000) // not finite
        return make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
    const uint64_t at = (uint64_t)(int64_t)position * turn_step(freq);
    const uint64_t quarter = (at + (1ull << 61)) >> 62; // nearest
    // The rest, up to pi / 4 either way, and the Taylor series of its sine up to x^9 and of its
    // cosine up to x^10: what is left out is below 2^-28.
    const float x = (float)(int64_t)(at - (quarter << 62)) * 3.4061215800304075e-19f; // 2 pi 2^-64
    const float z = x * x;
    float s = fmaf(z, fmaf(z, fmaf(z, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -1.6666667e-1f);
    s = fmaf(x * z, s, x);
    float c = fmaf(z, fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f);
    c = fmaf(z, fmaf(z, c, -0.5f), 1.f);
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

// Codes of eight values (the quantiser of pa_cache_write): the correctly rounded quotient
// x / scale, rounded to an integer, half to even. x times the reciprocal is off by less than
// 2^-14 (two roundings of up to 128), so where it is at least that far from a half both round
// to the same integer; the rest is divided, value by value: few, but half the largest value of
// a row, which bf16 rows often have, is 63.5 or 3.5 itself. Adding 1.5 * 2^23 rounds a small
// number to an integer, which the sum's low bits hold in two's complement (rint and the
// conversion run at an eighth of the rate). inv: 1 / scale, 0 where all codes are 0.
template <int KIND>
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float scale, float inv)
{
    constexpr float top = KIND == 1 ? 127.f : 7.f, kRound = 12582912.f;
    float c[8];
    uint32_t near = inv < 1e30f ? 0u : 0xffu; // (a scale near 0: all)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = x[i] * inv;
        c[i] = r + kRound;
        if (!(fabsf(r - (c[i] - kRound)) < 0.5f - 6.1035156e-5f)) // (or not a number)
            near |= 1u << i;
    }
#pragma unroll 1
    for (; near; near &= near - 1) {
        const int i = __ffs(near) - 1;
        float r = 0.f; // (x and c stay in registers: no index that is not a constant)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r = e == i ? x[e] : r;
        r = scale != 0.f ? fminf(fmaxf(rintf(__fdiv_rn(r, scale)), -top - 1.f), top) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e] = e == i ? r + kRound : c[e];
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = __float_as_uint(c[i]);
    if constexpr (KIND == 1)
        return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040),
                                      __byte_perm(w[2], w[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(w[4], w[5], 0x0040),
                                      __byte_perm(w[6], w[7], 0x0040), 0x5410));
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        n |= (w[i] & 0xfu) << (4 * i);
    return make_uint2(n, 0);
}

// KIND: 0 bf16, 1 INT8, 2 INT4; ADJ: pairs are adjacent values; U: pieces of a thread whose
// loads are in flight together
template <int D, int KIND, bool ADJ, int U>
__global__ void __launch_bounds__(kThreads, U == 1 ? 1 : 4) rope_write_kernel(const RopeParams p)
{
    // a decode launched next on the stream may be scheduled now; it waits for
    // this grid to complete before reading the cache
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int PPR = D / 16, STEP = kThreads / PPR; // pieces of a row, rows of a round
    extern __shared__ __align__(16) float2 turns[];    // [tokens][pairs]
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, p.num_tokens - t0);
    // this thread's piece of its rows: values from .. from + 7 and from + gap .. from + gap + 7
    const int c = tid % PPR;
    const bool turns_it = ADJ ? 16 * c < 2 * p.pairs : 8 * c < p.pairs;
    const int from = !ADJ && turns_it ? 8 * c : 16 * c, gap = !ADJ && turns_it ? p.pairs : 8;
    const float4 *cs = reinterpret_cast<const float4 *>(turns + (ADJ ? 8 * c : from));
    // row `row` of token `tok`, STEP rows further on from round to round
    int tok = 0, row = blockIdx.y * (STEP * U) + tid / PPR;
    if (row >= p.rows) {
        tok = row / p.rows;
        row -= tok * p.rows;
    }
    const int rounds = gridDim.y > 1 ? 1 : (tokens * p.rows + STEP * U - 1) / (STEP * U);
    for (int round = 0; round < rounds; ++round) {
        uint4 a[U], b[U];
        int64_t slot[U];
        int at_tok[U], at_row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool live = tok < tokens;
            at_tok[u] = live ? tok : -1;
            at_row[u] = row;
            const int64_t t = t0 + tok;
            const bool is_q = row < p.n_h, is_k = row < p.n_h + p.n_kv;
            const __nv_bfloat16 *src = is_q ? p.q : is_k ? p.k : p.v;
            const int64_t stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
            const int h = row - (is_q ? 0 : is_k ? p.n_h : p.n_h + p.n_kv);
            src += t * stride + h * D + from;
            a[u] = b[u] = make_uint4(0, 0, 0, 0);
            slot[u] = -1;
            if (live) {
                a[u] = *reinterpret_cast<const uint4 *>(src);
                b[u] = *reinterpret_cast<const uint4 *>(src + gap);
                if (!is_q)
                    slot[u] = p.slots[t];
            }
            row += p.round_rows;
            tok += p.round_tokens;
            if (row >= p.rows) {
                row -= p.rows;
                ++tok;
            }
        }
        if (round == 0) {
            for (int j = tid; j < tokens * p.pairs; j += kThreads) {
                const int t = j / p.pairs, i = j - t * p.pairs;
                const int axis = p.axis ? p.axis[i] : 0;
                float2 w = make_float2(1.f, 0.f); // (an axis that is not there turns nothing)
                if (axis >= 0 && axis < p.n_axes)
                    w = turn_of(p.positions[axis * p.num_tokens + t0 + t], p.inv_freq[i],
                                p.amplitude);
                else if (p.dev_status)
                    atomicOr(p.dev_status, PA_DEV_BAD_CONTEXT_BIT);
                turns[j] = w;
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool live = at_tok[u] >= 0;
            const bool is_q = at_row[u] < p.n_h, is_v = at_row[u] >= p.n_h + p.n_kv;
            float x[8], y[8];
            if (KIND != 0 || !is_v) {
                unpack(a[u], x);
                unpack(b[u], y);
            }
            if (live && turns_it && !is_v) {
                const float4 *w4 = cs + at_tok[u] * (p.pairs / 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) { // two pairs at a time
                    const float4 w = w4[e];
                    float *m = ADJ ? (e < 2 ? x + 4 * e : y + 4 * (e - 2)) : x + 2 * e;
                    float *n = ADJ ? m + 1 : y + 2 * e;
                    constexpr int next = ADJ ? 2 : 1;
                    const float a0 = m[0], b0 = n[0], a1 = m[next], b1 = n[next];
                    m[0] = a0 * w.x - b0 * w.y;
                    n[0] = b0 * w.x + a0 * w.y;
                    m[next] = a1 * w.z - b1 * w.w;
                    n[next] = b1 * w.z + a1 * w.w;
                }
            }
            if ((KIND == 0 || is_q) && !is_v) {
                a[u] = pack(x);
                b[u] = pack(y);
            }
            if (live && is_q) {
                __nv_bfloat16 *dst =
                    p.out + ((t0 + at_tok[u]) * p.n_h + at_row[u]) * D + from;
                *reinterpret_cast<uint4 *>(dst) = a[u];
                *reinterpret_cast<uint4 *>(dst + gap) = b[u];
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
            if (is_q || !live)
                continue;
            const int64_t s = slot[u];
            const int h = at_row[u] - p.n_h - (is_v ? p.n_kv : 0);
            const bool lead = c == 0;
            if (s < 0 || s >= p.num_slots) {
                if (s >= 0 && lead && h == 0 && p.dev_status)
                    atomicOr(p.dev_status, PA_DEV_BAD_SLOT_BIT);
                continue;
            }
            const int64_t dst_row = ((s >> 4) * p.n_kv + h) * 16 + (s & 15);
            void *pool = is_v ? p.v_cache : p.k_cache;
            if constexpr (KIND == 0) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(pool) + dst_row * D + from;
                *reinterpret_cast<uint4 *>(dst) = a[u];
                *reinterpret_cast<uint4 *>(dst + gap) = b[u];
            } else {
                const float inv = scale != 0.f ? __frcp_rn(scale) : 0.f;
                const uint2 cx = codes_of<KIND>(x, scale, inv), cy = codes_of<KIND>(y, scale, inv);
                if constexpr (KIND == 1) {
                    int8_t *dst = static_cast<int8_t *>(pool) + dst_row * D + from;
                    *reinterpret_cast<uint2 *>(dst) = cx;
                    *reinterpret_cast<uint2 *>(dst + gap) = cy;
                } else {
                    uint8_t *dst = static_cast<uint8_t *>(pool) + (dst_row * D + from) / 2;
                    *reinterpret_cast<uint32_t *>(dst) = cx.x;
                    *reinterpret_cast<uint32_t *>(dst + gap / 2) = cy.x;
                }
                if (lead)
                    (is_v ? p.v_scale : p.k_scale)[dst_row] = scale;
            }
        }
    }
}

template <int D, int KIND, bool ADJ>
cudaError_t launch_of(const RopeParams &p, int sms, cudaStream_t stream)
{
    constexpr int STEP = kThreads / (D / 16);
    RopeParams r = p;
    const int64_t rounds = (p.rows + STEP - 1) / STEP; // of one token alone
    if (p.num_tokens * rounds <= 2 * sms) {            // few: a round to a CTA
        r.tokens = 1;
        r.round_rows = 0;
        r.round_tokens = 1; // the one round is the last
        rope_write_kernel<D, KIND, ADJ, 1>
            <<<dim3((unsigned)p.num_tokens, (unsigned)rounds), kThreads,
               p.pairs * sizeof(float2), stream>>>(r);
    } else {
        // Tokens of a CTA, up to four sines and cosines to a thread: the fewest rounds, those of
        // the sines included, over all waves of four CTAs to an SM (4 + 1 heads of 128, 30000
        // tokens: 25 us against 34 with four tokens).
        int64_t best = INT64_MAX;
        for (int t = 1; t <= 4 * kThreads / p.pairs; ++t) {
            const int64_t waves = (p.num_tokens + (int64_t)t * 4 * sms - 1) / ((int64_t)t * 4 * sms);
            const int64_t cost = waves * (((int64_t)t * p.rows + 2 * STEP - 1) / (2 * STEP) +
                                          (t * p.pairs + kThreads - 1) / kThreads);
            if (cost < best) {
                best = cost;
                r.tokens = t;
            }
        }
        r.round_rows = STEP % p.rows;
        r.round_tokens = STEP / p.rows;
        const int64_t blocks = (p.num_tokens + r.tokens - 1) / r.tokens;
        if (blocks > 0x7fffffff)
            return cudaErrorInvalidValue;
        rope_write_kernel<D, KIND, ADJ, 2>
            <<<(unsigned)blocks, kThreads, r.tokens * p.pairs * sizeof(float2), stream>>>(r);
    }
    return cudaGetLastError();
}

template <int D, int KIND>
cudaError_t launch_of(const RopeParams &p, bool adjacent, int sms, cudaStream_t stream)
{
    return adjacent ? launch_of<D, KIND, true>(p, sms, stream)
                    : launch_of<D, KIND, false>(p, sms, stream);
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
    p.rows = a.n_h + 2 * a.n_kv;
    p.tokens = 1;
    p.round_rows = p.round_tokens = 0;
    if (a.d_h == 128)
        return a.kind == 0   ? launch_of<128, 0>(p, a.adjacent != 0, sms, stream)
               : a.kind == 1 ? launch_of<128, 1>(p, a.adjacent != 0, sms, stream)
                             : launch_of<128, 2>(p, a.adjacent != 0, sms, stream);
    return a.kind == 0   ? launch_of<64, 0>(p, a.adjacent != 0, sms, stream)
           : a.kind == 1 ? launch_of<64, 1>(p, a.adjacent != 0, sms, stream)
                         : launch_of<64, 2>(p, a.adjacent != 0, sms, stream);
}

} // namespace pa
