// Cross attention: any number of query tokens per sequence over a paged K/V cache
// of another length (an encoder's states, or rows an eviction kept).
//
//     s_j = scale <q[t][h], K_b[j][h / g]>,  j < ctx_b (no mask)
//     out[t][h] = sum_j softmax(s)_j V_b[j][h / g],  cu_q[b] <= t < cu_q[b + 1]
//
// What bounds it: 4 d_h FLOP per (query row, key) against 2 rows of K/V bytes per
// (kv head, key). A tile of 256 query rows is past the ridge (the tensor cores
// bound it), a few rows leave it at the K/V stream.
//
// Split. The query rows of a kv head (tokens x the g heads that share it) are
// packed: row t * g + h. A unit is (sequence, kv head, up to 256 packed rows),
// one or two halves of 128 rows = one tensor-core tile each; its items are
// the 128-key tiles of the context. Items lie on one line, as long as they take
// (kWeight), and CTA c of G takes [c W / G, (c + 1) W / G) of it, so any mix of
// lengths is balanced and a few long contexts still use every SM. A unit cut
// by CTA borders leaves (m, l, O) records; the last CTA to finish it merges them
// (log-sum-exp). No CTA waits for another.
//
// One CTA per SM, 12 warps (16 for INT8/INT4):
//   warps 0-3, 4-7  softmax of buffer 0 and buffer 1, a thread per query row
//   warp 8          issues the matrix instructions (one thread)
//   warp 9          copies of Q and of the paged K/V blocks: TMA boxes of 16 rows x 64
//                   columns in the 128-byte swizzle; codes and scales as bulk copies
//   warps 10-15     INT8/INT4 pools: write the codes that warp 9 copies as bf16
//                   (exact: 8 significant bits) into the same tiles; the K
//                   scale multiplies the scores, the V scale the weights
// Tensor memory (512 columns): two buffers of scores (128 fp32 columns) and of outputs
// (d_h columns). The weights P overwrite their scores as two bf16 parts each, what rounding
// leaves of the first in the second, and both are A operands of P V: 2^-16 relative per
// weight. With the first part alone (2^-8) rows of V that span 1e-3 .. 1e3 and cancel leave
// the decode's tolerance of 1e-2 (1 + |out|). It costs half as many products again and the
// forming of the second parts: prompts 465 -> 617 us and up, mixed batch 105 -> 121, INT8
// 198 -> 230. Sums l take the unrounded weights. A unit of two halves gives each a buffer;
// one of one half uses both in turn, tile after tile, and joins its two states at the end.
// So one buffer is in its softmax while the other has the tensor cores.
//
// The softmax base of a row moves rarely (kMoveLog2), so O is rarely rescaled.
//
// Measured on a GB300 (g = 4, d_h 128, bf16): 8 prompts of 512..1024 tokens over
// 4096..8192 keys 616 us (680 back to back, under the power cap), 1030 TFLOP/s with each
// product counted once, 0.53 of the measured bf16 matrix rate; a buffer's chain (the last
// 64 keys' products, 290 cycles until they are seen, scores 512, softmax) bounds a tile of
// 256 x 128 at 4650 cycles against about 3100 of products. 48 sequences of 1..61 tokens over
// 200..4096 keys 121 us, 3690 GB/s, 0.54 of the measured copy rate: the same chain, first
// loads, unit ends and merges.
#include "pa_decode.cuh"
#include "pa_launch.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kMmaWarp = 8, kCopyWarp = 9;
constexpr int kRows = 128;       // query rows of a half, keys of a tile
constexpr int kTileBlocks = kRows / kBlockTokens;
constexpr int kPart = kRows / 2; // keys of one softmax step
// What an item takes, of a unit of two halves and of one: 4 : 3 against 1 : 1 and 2 : 1 in us:
// the mixed batch 121 / 130 / 135, INT8 230 / 242 / 267, heads of 64 103 / 110 / 97.
constexpr int kWeight2 = 4, kWeight1 = 3;
// ... and each unit, in front of its first item, for its queries and outputs.
constexpr int kUnitCost = 5;
constexpr int kUnitRows = 2 * kRows;
constexpr int kConvWarps = 6;    // INT8/INT4: warps that turn codes into bf16
constexpr int kScaleRing = 8;    // tiles whose scales are kept (at most five live)
// A row's softmax base moves only when a step's maximum exceeds it by more than this: exact,
// since P, l and O share one base and weights up to 2^16 are as exact in bf16 as those up to 1
// (the sums stay finite for |V| below 2^90). A move costs about 2000 cycles, the wait for the
// products so far included: with 2^8 the INT8 batch took 242 us, with 2^16 221.
constexpr float kMoveLog2 = 16.f;

struct CrossParams {
    const void *k_cache;
    const void *v_cache;
    const float *k_scale;
    const float *v_scale;
    const int32_t *cu_q;
    const int32_t *block_tables;
    const int32_t *context_lens;
    __nv_bfloat16 *out;
    float *records;    // [num_ctas][2], see record_floats
    int32_t *counters; // [num_ctas], zero between calls
    int32_t *dev_status;
    int64_t num_q;
    int64_t num_blocks;
    int32_t num_seqs;
    int32_t n_kv;
    int32_t log2_g;  // of the query heads per kv head
    int32_t max_blocks;
    int32_t num_ctas;
    float scale_log2;
};

struct Seq {
    int32_t ctx, q0, nq;
    int32_t tiles;  // 128-key tiles
    int32_t pairs;  // units of one kv head's packed query rows with two halves,
    int32_t units;  // and all of them (the last may have one)
    __device__ int64_t head() const // positions of one kv head
    {
        const int64_t items = kWeight2 * (int64_t)pairs + kWeight1 * (units - pairs);
        return tiles == 0 ? 0 : tiles * items + (int64_t)kUnitCost * units;
    }
    __device__ int64_t length(const CrossParams &p) const { return p.n_kv * head(); }
};

// Sequence b's sizes; bad ones (reported where `report`) count as nothing.
__device__ __forceinline__ Seq load_seq(const CrossParams &p, int b, bool report)
{
    Seq s;
    const int32_t ctx = __ldg(p.context_lens + b);
    const int32_t q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    const bool q_ok = q0 >= 0 && q1 >= q0 && q1 <= p.num_q;
    const bool c_ok = ctx >= 0 && ctx <= (int64_t)p.max_blocks * kBlockTokens;
    if (report && (!q_ok || !c_ok))
        flag_error(p.dev_status, PA_DEV_BAD_CONTEXT_BIT);
    s.ctx = c_ok ? ctx : 0;
    s.q0 = q_ok ? q0 : 0;
    s.nq = q_ok ? q1 - q0 : 0;
    s.tiles = (int32_t)(((int64_t)s.ctx + kRows - 1) / kRows);
    const int64_t halves = (((int64_t)s.nq << p.log2_g) + kRows - 1) / kRows;
    s.pairs = (int32_t)(halves / 2);
    s.units = (int32_t)((halves + 1) / 2);
    return s;
}

// A run of items of one unit that this CTA takes.
struct Segment {
    int kvh;
    int halves;      // 1 or 2
    int64_t row0;    // first packed row of the unit within (sequence, kv head)
    int rows;        // live rows: 1 .. 256
    int j0, j1;      // key tiles [j0, j1)
    int64_t first_v; // the position of the unit's first item
    int weight;      // positions of one item
    bool whole;
};

// The first item a CTA owns: an item belongs to the CTA with its first position.
struct Start {
    int64_t pos;
    int32_t b, kvh, qt, j; // sequence, kv head, unit of that head, key tile
};

// The segments of the items at positions [start, hi) of the line, one after another.
struct Walk {
    const CrossParams &p;
    int64_t hi;
    Start at;
    Seq s;

    __device__ Walk(const CrossParams &p_, int64_t hi_, const Start &at_)
        : p(p_), hi(hi_), at(at_), s(load_seq(p_, at_.b, false))
    {
    }

    __device__ bool next(Segment &g)
    {
        if (at.pos >= hi)
            return false;
        if (at.qt == s.units) {
            at.qt = 0;
            if (++at.kvh == p.n_kv) {
                at.kvh = 0;
                do // (below the line's end there is a sequence with items)
                    s = load_seq(p, ++at.b, false);
                while (s.tiles == 0 || s.units == 0);
            }
        }
        g.halves = at.qt < s.pairs ? 2 : 1;
        g.weight = g.halves == 2 ? kWeight2 : kWeight1;
        const int64_t room = div_small(hi - at.pos + g.weight - 1, g.weight);
        const int n = (int)min((int64_t)(s.tiles - at.j), room);
        g.kvh = at.kvh;
        g.j0 = at.j;
        g.j1 = at.j + n;
        g.first_v = at.pos - (int64_t)at.j * g.weight;
        g.row0 = (int64_t)at.qt * kUnitRows;
        g.rows = (int)min((int64_t)kUnitRows, ((int64_t)s.nq << p.log2_g) - g.row0);
        g.whole = n == s.tiles;
        at.pos += (int64_t)n * g.weight + kUnitCost; // (to the next unit's first item)
        at.j = 0;
        ++at.qt;
        return true;
    }
};

// A record: O as float4 [d / 4][row], then (m, l) per row; coalesced for a thread per row.
constexpr int record_floats(int d) { return kUnitRows * (d + 2); }

// Log-sum-exp state of eight adjacent outputs of one row.
struct MergeState {
    float m, l, o[8];
    __device__ __forceinline__ void clear()
    {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] = 0.f;
    }
    // Outputs 8 d8 .. 8 d8 + 7 of row `row` of one or two (r1 not NULL) records.
    template <int D>
    __device__ __forceinline__ void fold(const float *r0, const float *r1, int row, int d8)
    {
        float2 ml[2];
        float4 x[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float *r = k ? r1 : r0;
            ml[k] = make_float2(-INFINITY, 0.f);
            x[k][0] = x[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r) {
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(r + D * kUnitRows) + row);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x[k][e] = __ldcg(reinterpret_cast<const float4 *>(r) +
                                     (2 * d8 + e) * kUnitRows + row);
            }
        }
        const float top = fmaxf(m, fmaxf(ml[0].x, ml[1].x));
        if (top == -INFINITY)
            return;
        const float a = fast_exp2(m - top);
        m = top;
        l *= a;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] *= a;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float f = fast_exp2(ml[k].x - top);
            l = fmaf(f, ml[k].y, l);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                o[4 * e] = fmaf(f, x[k][e].x, o[4 * e]);
                o[4 * e + 1] = fmaf(f, x[k][e].y, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(f, x[k][e].z, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(f, x[k][e].w, o[4 * e + 3]);
            }
        }
    }
};

// CTAs that take part: each range is as long as the longest item. So a range that lies between
// the first positions of a unit's first and last item holds an item's first position: every CTA
// from the first item's owner to the last one's has an item of the unit, and each of them
// leaves a record and arrives. A range that lies within a unit's charge owns nothing.
static_assert(kWeight2 >= kWeight1, "the longest item");
__device__ __forceinline__ int64_t line_ctas(const CrossParams &p, int64_t total)
{
    return total == 0 ? 0 : max((int64_t)1, plan_ctas(p.num_ctas, total / kWeight2));
}

template <int D, int KIND>
struct Smem {
    static constexpr int TILE = kRows * D * 2; // one Q half, K tile or V tile in bf16
    static constexpr int kThreads = KIND ? (kCopyWarp + 1 + kConvWarps) * 32 : 384;
    // tiles in bf16, and (INT8/INT4) tiles of codes on their way
    static constexpr int SLOTS = (KIND ? 3 : 4) * (128 / D);
    static constexpr int ROWB = KIND == 1 ? D : D / 2;
    static constexpr int RAW = kRows * ROWB + 2 * kRows * 4; // codes, K and V scales
    static constexpr int RAWS = KIND == 0 ? 0 : KIND == 1 ? SLOTS : 6;
    static constexpr int kOffRing = 2 * TILE;
    static constexpr int kOffScales = kOffRing + SLOTS * TILE; // [ring][K, V][128] fp32
    static constexpr int kScaleBytes = KIND ? kScaleRing * 2 * kRows * 4 : 0;
    static constexpr int kOffRaw = kOffScales + kScaleBytes;
    static constexpr int kOffBars = kOffRaw + RAWS * RAW;
    static constexpr int kBars = 2 + 2 * SLOTS + 10 + 1 + 2 * RAWS;
    static constexpr int kOffMisc = kOffBars + (kBars * 8 + 15) / 16 * 16; // 64 int32
    static constexpr int kOffRows = kOffMisc + 256; // (m, l) [buffer][128]
    static constexpr int kBytes = 1024 + kOffRows + 2 * kRows * 8;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tmap, int32_t x,
                                            int32_t y, int32_t z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4])
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ void bar_named(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Two fp32 lanes per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}

// Two weights in two bf16 parts each: hi rounds them, lo rounds what is left of them (exact in
// fp32), 2^-16 relative together.
__device__ __forceinline__ void split_bf16x2(float2 x, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x.x, x.y);
    const float2 r = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                          make_float2(-1.f, -1.f), x);
    lo = pack_bf16x2(r.x, r.y);
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two INT8 codes (bytes SEL picks, zero-extended to 16 bits) as bf16, exactly:
// 0x4300 | low 7 bits is 128 + those bits, 0x4300 | sign bit is 128 or 256.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t code8_bf2(uint32_t x)
{
    const uint32_t w = __byte_perm(x, 0, SEL);
    return sub_bf16x2((w & 0x007f007fu) | 0x43004300u, (w & 0x00800080u) | 0x43004300u);
}

// The two INT4 codes of byte K of the word whose low nibbles are a and high
// nibbles b, offset by 8: 0x4300 | n is 128 + n, and 0x4308 is 136.
template <int K>
__device__ __forceinline__ uint32_t code4_bf2(uint32_t a, uint32_t b)
{
    const uint32_t t = __byte_perm(a, b, K | (K << 4) | ((4 + K) << 8) | ((4 + K) << 12));
    return sub_bf16x2((t & 0x000f000fu) | 0x43004300u, 0x43084308u);
}

// mbar_wait whose polling is a few instructions: unrolled, as the compiler would, the
// waiting warps' polls push the working ones' code out of the instruction cache.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (i % 64 == 0 && global_timer_ns() - t0 > 1000000000ull)
            return false; // about a second: give up, as mbar_wait does
    }
}

// The same with the polling out of line, for the thread that issues the matrix
// instructions: its waits are mostly over when it comes to them.
__device__ __noinline__ bool mbar_poll_slow(uint32_t bar, uint32_t parity)
{
    return mbar_poll(bar, parity);
}
__device__ __forceinline__ bool mbar_ready(uint32_t bar, uint32_t parity)
{
    return mbar_try_wait(bar, parity) || mbar_poll_slow(bar, parity);
}

// One step of the online softmax over 64 keys of an INT8/INT4 tile, of a warp's 32 rows. A
// thread has four rows, lane / 4 + 8 i, and two of every eight keys: each scale that it loads
// serves four rows: 16 loads of 8 bytes a step where a row per thread takes 32 of 16 (the INT8
// batch in 213 us against 221).
//   sk      K scales of the keys, V scales kRows behind
//   here    keys of the step within the context; bad: its bad blocks, -1: no key is masked
//   wait_o  O is complete
template <int D, class WaitO>
__device__ __forceinline__ void quad_step(uint32_t tS, uint32_t tO, const float *sk, int c0,
                                          int here, int bad, bool first, float (&m)[4],
                                          float (&l)[4], WaitO wait_o)
{
    constexpr uint32_t kUpper = 16u << 16; // lanes 16 .. 31
    const int lane = threadIdx.x & 31, c2 = 2 * (lane & 3);
    float s[kPart]; // [i / 2][8 keys k][i % 2][2]
    tmem_ld_quad(tS + c0, s);
    tmem_ld_quad(tS + kUpper + c0, s + 32);
    tmem_wait_ld();
    tmem_landed<kPart>(s);
    sk += c2;
    auto at = [](int i, int k) { return (i / 2) * 32 + 4 * k + 2 * (i % 2); };
#pragma unroll
    for (int k = 0; k < 8; ++k) { // scores in the log2 domain
        const float2 f = *reinterpret_cast<const float2 *>(sk + 8 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = mul2(make_float2(s[at(i, k)], s[at(i, k) + 1]), f);
            s[at(i, k)] = x.x;
            s[at(i, k) + 1] = x.y;
        }
    }
    if (bad >= 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool block = (bad >> (k / 2)) & 1;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (block || 8 * k + c2 + e >= here)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[at(i, k) + e] = -INFINITY;
        }
    }
    float top[4];
    bool up = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        top[i] = fmaxf(s[at(i, 0)], s[at(i, 0) + 1]);
#pragma unroll
        for (int k = 1; k < 8; ++k)
            top[i] = max3(top[i], s[at(i, k)], s[at(i, k) + 1]);
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        if (first)
            m[i] = top[i];
        up = up || top[i] > m[i] + kMoveLog2;
    }
    if (__any_sync(0xffffffffu, up)) {
        wait_o();
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool move = top[i] > m[i] + kMoveLog2;
            a[i] = move ? fast_exp2(m[i] - top[i]) : 1.f;
            m[i] = move ? top[i] : m[i];
            l[i] *= a[i];
        }
#pragma unroll 1
        for (int c = 0; c < 2 * D; c += 64) { // columns c % D of the lower, then the upper lanes
            const float a0 = c < D ? a[0] : a[2], a1 = c < D ? a[1] : a[3];
            const uint32_t addr = tO + (c < D ? (uint32_t)c : kUpper + (uint32_t)(c - D));
            float o[32];
            tmem_ld_quad(addr, o);
            tmem_wait_ld();
            tmem_landed<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                o[e] *= e & 2 ? a1 : a0;
            tmem_st_quad(addr, o);
        }
    }
    float2 base[4], sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = m[i] == -INFINITY ? 0.f : -m[i];
        base[i] = make_float2(x, x);
        sum[i] = make_float2(0.f, 0.f);
    }
    uint32_t w[2][16], low[2][16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 f = *reinterpret_cast<const float2 *>(sk + kRows + 8 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 x = add2(make_float2(s[at(i, k)], s[at(i, k) + 1]), base[i]);
            x.x = fast_exp2(x.x);
            x.y = fast_exp2(x.y);
            sum[i] = add2(sum[i], x);
            split_bf16x2(mul2(x, f), w[i / 2][2 * k + i % 2], low[i / 2][2 * k + i % 2]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t at_lanes = tS + (i ? kUpper : 0u) + c0;
        tmem_st_quad_bf16(at_lanes, w[i]);
        tmem_st_quad_bf16(at_lanes + kPart / 2, low[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        l[i] += sum[i].x + sum[i].y;
}

template <int D, int KIND>
__global__ void __launch_bounds__(Smem<D, KIND>::kThreads, 1)
cross_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const CrossParams p)
{
    using L = Smem<D, KIND>;
    constexpr int kThreads = L::kThreads, SLOTS = L::SLOTS, TILE = L::TILE, HALVES = D / 64;
    constexpr int COL = TILE / HALVES; // bytes of one 64-element column of a tile
    constexpr int RECORD = record_floats(D);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t ring = sbase + L::kOffRing;
    const uint32_t bars = sbase + L::kOffBars;
    const uint32_t q_full = bars, q_empty = bars + 8, kv_full = bars + 16,
                   kv_empty = kv_full + 8 * SLOTS, s_full = kv_empty + 8 * SLOTS,
                   p_full = s_full + 16 /* [half][part] */, o_full = p_full + 32,
                   a_full = o_full + 16, drained = a_full + 16, raw_full = drained + 8,
                   raw_empty = raw_full + 8 * L::RAWS;
    // misc: [0] tensor memory base (0), [1] merge flag, [2..7] the CTA's first item,
    // [8..] bad-block masks per slot, [16..17] per half, [18..23] blocks of
    // the tiles of codes, [24..] scan
    int32_t *misc = reinterpret_cast<int32_t *>(smem + L::kOffMisc);
    volatile int32_t *slot_mask = misc + 8;
    volatile int32_t *half_mask = misc + 16;
    volatile int32_t *raw_mask = misc + 18; // present blocks | bad ones << 8

    auto record = [&](int64_t i) { return p.records + i * RECORD; };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_h = p.n_kv << p.log2_g, g_mask = (1 << p.log2_g) - 1;

    // ---- this CTA's range of the line
    int64_t total;
    {
        const int per = (p.num_seqs + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, p.num_seqs), b1 = min(b0 + per, p.num_seqs);
        int64_t sum = 0;
        for (int b = b0; b < b1; ++b)
            sum += load_seq(p, b, blockIdx.x == 0).length(p);
        int64_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        int64_t *wsum = reinterpret_cast<int64_t *>(misc + 24);
        if (lane == 31)
            wsum[warp] = x;
        __syncthreads();
        int64_t before = x - sum;
        total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            before += w < warp ? wsum[w] : 0;
            total += wsum[w];
        }
        if (total > 0) {
            const int64_t G = line_ctas(p, total);
            const int64_t lo = plan_lo(blockIdx.x, total, G);
            if (blockIdx.x < G && lo >= before && lo < before + sum) {
                int b = b0;
                int64_t v = before;
                Seq q = load_seq(p, b, false);
                while (lo >= v + q.length(p)) { // (one of the thread's sequences holds lo)
                    v += q.length(p);
                    q = load_seq(p, ++b, false);
                }
                const int64_t head = q.head(), kvh = div_small(lo - v, head);
                const int64_t in = lo - v - kvh * head;
                const int64_t pair = (int64_t)q.tiles * kWeight2 + kUnitCost;
                const int64_t qt = min(div_small(in, pair), (int64_t)q.pairs);
                const int64_t weight = qt < q.pairs ? kWeight2 : kWeight1;
                // from the unit's first item on
                const int64_t off = max(in - qt * pair - kUnitCost, (int64_t)0);
                const int64_t j = div_small(off + weight - 1, weight);
                const bool past = j == q.tiles; // within the unit's last item: on to the next
                const int64_t first_v = v + kvh * head + qt * pair + kUnitCost;
                *reinterpret_cast<Start *>(misc + 2) = {
                    first_v + j * weight + (past ? kUnitCost : 0), b, (int32_t)kvh,
                    (int32_t)(past ? qt + 1 : qt), (int32_t)(past ? 0 : j)};
            }
        }
    }
    // sequences without keys: zero rows (threads t of n)
    auto zero_rows = [&](int t, int n) {
        for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x) {
            const Seq q = load_seq(p, b, false);
            if (q.nq > 0 && q.tiles == 0) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + (int64_t)q.q0 * n_h * D);
                const int64_t chunks = (int64_t)q.nq * n_h * (D / 8);
                for (int64_t i = t; i < chunks; i += n)
                    dst[i] = make_uint4(0, 0, 0, 0);
            }
        }
    };
    const int64_t G = line_ctas(p, total);
    if (blockIdx.x >= G) { // (no items: no CTA)
        zero_rows(tid, kThreads);
        return;
    }
    const int64_t hi = plan_lo(blockIdx.x + 1, total, G);

    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(kv_full + 8 * s, KIND ? kConvWarps : 1);
            mbar_init(kv_empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 2); // the matrix instructions and the mask
            mbar_init(p_full + 16 * i, kRows);
            mbar_init(p_full + 16 * i + 8, kRows);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(a_full + 8 * i, 1);
        }
        mbar_init(drained, 1);
        for (int s = 0; s < L::RAWS; ++s) {
            mbar_init(raw_full + 8 * s, 1);
            mbar_init(raw_empty + 8 * s, kConvWarps);
        }
        fence_barrier_init();
    }
    if (warp == kMmaWarp)
        tmem_alloc(smem_u32(misc), 512); // all of it: its base address is 0
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;
    Walk walk(p, hi, *reinterpret_cast<const Start *>(misc + 2));
    Segment g;
    bool dead = false; // a wait gave up: no more waits, no more copies or products
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!dead && !__all_sync(0xffffffffu, mbar_poll(bar, parity & 1u))) {
            dead = true;
            if (lane == 0)
                flag_error(p.dev_status, PA_DEV_TIMEOUT_BIT);
        }
        return !dead;
    };

    if (warp < kMmaWarp) {
        // ================================================================ softmax
        if constexpr (KIND != 0) { // 256 x 160 + 256 x 96 = the 512 x 128 of the launch
            static_assert(kThreads == 512, "whole groups of four warps share registers");
            asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        }
        const int half = warp >> 2;
        const int row = tid & (kRows - 1);
        // (m, l) of each buffer's rows, where the two buffers share a half's rows
        float2 *states = reinterpret_cast<float2 *>(smem + L::kOffRows);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21; // lane base of this warp, bits 16..
        const uint32_t tS = tmem + lanes + half * 128, tO = tmem + lanes + 256 + half * 128;
        const float *scales = reinterpret_cast<const float *>(smem + L::kOffScales);
        uint32_t n_b[2] = {0, 0}; // tiles of each buffer so far
        uint32_t n_tile = 0;  // tiles of this CTA so far (the scale ring's index)
        while (walk.next(g)) {
            const int ctx = walk.s.ctx;
            // this thread's row (INT8/INT4: its four rows, see there)
            constexpr int kOwn = KIND ? 4 : 1;
            float ms[kOwn], ls[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                ms[i] = -INFINITY;
                ls[i] = 0.f;
            }
            // two halves: each buffer one half, every tile; one half: both buffers its rows,
            // every other tile
            const bool two = g.halves == 2;
            const int j_first = two ? g.j0 : g.j0 + half, step = two ? 1 : 2;
            uint32_t n_s = half ? n_b[1] : n_b[0];
            for (int j = j_first; j < g.j1; j += step, ++n_s) {
                if (!wait(s_full + 8 * half, n_s))
                    break;
                tc_fence_after();
                const int bad = half_mask[half];
                const int valid = min(ctx - j * kRows, kRows);
                const float *sk =
                    scales + ((n_tile + (uint32_t)(j - g.j0)) % kScaleRing) * 2 * kRows;
                const int tail = ctx % kBlockTokens;
                if (KIND == 0 && tail && j == walk.s.tiles - 1) {
                    // V rows behind the context may hold anything, and 0 * NaN is NaN: zero
                    // them before this half's products (both halves write the same zeros)
                    const uint32_t fill = 2 * (n_tile + (uint32_t)(j - g.j0)) + 1;
                    const uint32_t v_at = ring + fill % SLOTS * TILE;
                    if (wait(kv_full + 8 * (fill % SLOTS), fill / SLOTS))
                        for (int i = tid & (kRows - 1); i < (kBlockTokens - tail) * (D / 8);
                             i += kRows) {
                            const int rr = valid + i / (D / 8), c = i % (D / 8);
                            sts128(v_at + (c / 8) * COL + rr * 128 + (c % 8) * 16, 0, 0, 0, 0);
                        }
                    fence_proxy_async_smem();
                }
                // The tile's two halves of 64 keys are two steps of the online softmax: the
                // products of the first start while the weights of the second are formed.
                // (One copy of the code for both: unrolled, the kernel's loops no longer fit the
                // instruction cache together.)
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    const int c0 = part * kPart;
                    const bool first = part == 0 && j == j_first;
                    if constexpr (KIND != 0) {
                        quad_step<D>(tS, tO, sk + c0, c0, valid - c0,
                                     valid < kRows || bad ? bad >> (c0 / kBlockTokens) : -1, first,
                                     ms, ls, [&]() {
                                         if (part == 1) {
                                             wait(a_full + 8 * half, n_s);
                                             tc_fence_after();
                                         }
                                     });
                    } else {
                        float &m = ms[0], &l = ls[0];
                        float s[kPart];
                        tmem_ld32(tS + c0, s);
                        tmem_ld32(tS + c0 + 32, s + 32);
                        tmem_wait_ld();
                        tmem_landed<kPart>(s);
                        // scores in the log2 domain = s * mul
                        float mul = p.scale_log2;
                        if (valid < kRows || bad || mul < 0.f) {
                            const int here = valid - c0, bad_here = bad >> (c0 / kBlockTokens);
#pragma unroll
                            for (int c = 0; c < kPart; ++c)
                                s[c] = c < here && !((bad_here >> (c / kBlockTokens)) & 1)
                                           ? s[c] * mul
                                           : -INFINITY;
                            mul = 1.f;
                        }
                        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int c = 4; c < kPart - 4; c += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mx[e] = max3(mx[e], s[c + e], s[c + 4 + e]);
                        const float *end = s + kPart - 4;
                        const float top = mul * fmaxf(max3(mx[0], end[0], end[1]),
                                                      fmaxf(max3(mx[1], end[2], end[3]),
                                                            fmaxf(mx[2], mx[3])));
                        if (first) {
                            m = top;
                        } else {
                            const bool up = top > m + kMoveLog2;
                            if (__any_sync(0xffffffffu, up)) {
                                // O holds every earlier tile, and in the second step the first's
                                // products, once they are done
                                if (part == 1) {
                                    wait(a_full + 8 * half, n_s);
                                    tc_fence_after();
                                }
                                const float a = up ? fast_exp2(m - top) : 1.f;
                                m = up ? top : m;
                                l *= a;
#pragma unroll 1
                                for (int c = 0; c < D; c += 32) {
                                    float o[32];
                                    tmem_ld32(tO + c, o);
                                    tmem_wait_ld();
                                    tmem_landed<32>(o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        o[e] *= a;
                                    tmem_st32(tO + c, reinterpret_cast<const uint32_t *>(o));
                                }
                            }
                        }
                        const float base = m == -INFINITY ? 0.f : m;
                        const float2 mul_2 = make_float2(mul, mul);
                        const float2 base_2 = make_float2(-base, -base);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        uint32_t w[32], low[32];
#pragma unroll
                        for (int e = 0; e < kPart; e += 4) {
                            float2 x[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int at = e + 2 * i;
                                x[i] = fma2(make_float2(s[at], s[at + 1]), mul_2, base_2);
                                x[i].x = fast_exp2(x[i].x);
                                x[i].y = fast_exp2(x[i].y);
                                sum[i] = add2(sum[i], x[i]);
                            }
                            split_bf16x2(x[0], w[e / 2], low[e / 2]);
                            split_bf16x2(x[1], w[e / 2 + 1], low[e / 2 + 1]);
                        }
                        tmem_st32(tS + c0, w);
                        tmem_st32(tS + c0 + kPart / 2, low);
                        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full + 16 * half + 8 * part);
                }
            }
            const int n = g.j1 - g.j0;
            n_tile += (uint32_t)n;
            n_b[0] += two ? n : (n + 1) / 2;
            n_b[1] += two ? n : n / 2;
            // ---- the half's output, or its record
            const int r = two ? half * kRows + row : row; // row within the unit
            const bool live = r < g.rows;
            const int64_t prow = g.row0 + r; // packed row of (sequence, kv head)
            __nv_bfloat16 *o_row =
                p.out + ((walk.s.q0 + (prow >> p.log2_g)) * n_h + (g.kvh << p.log2_g) +
                         (prow & g_mask)) * D;
            float *rec = record((int64_t)blockIdx.x * 2 + (g.j0 > 0 ? 0 : 1));
            // 32 outputs from column c on, of a row whose weights sum to l
            auto emit = [&](int c, const float (&o)[32], float inv) {
                if (live && g.whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4 *>(o_row + c + e) =
                            make_uint4(pack_bf16x2(o[e] * inv, o[e + 1] * inv),
                                       pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                       pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv),
                                       pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        reinterpret_cast<float4 *>(rec)[(c + e) / 4 * kUnitRows + r] =
                            make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            };
            // (a sum that is not a number must not be skipped for its base)
            float m = ls[0] != ls[0] ? 0.f : ms[0], l = ls[0];
            if constexpr (KIND != 0) { // from the quads to a row per thread
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    float x = ls[i];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if ((lane & 3) == 0)
                        states[half * kRows + (row & ~31) + 8 * i + lane / 4] =
                            make_float2(x != x ? 0.f : ms[i], x);
                }
                __syncwarp();
                m = states[half * kRows + row].x;
                l = states[half * kRows + row].y;
            }
            if (two) {
                wait(o_full + 8 * half, n_s - 1);
                tc_fence_after();
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
                for (int c = 0; !dead && c < D; c += 32) {
                    float o[32];
                    tmem_ld32(tO + c, o);
                    tmem_wait_ld();
                    tmem_landed<32>(o);
                    emit(c, o, inv);
                }
            } else {
                // both buffers' states of this row join; each thread takes half the columns
                if constexpr (KIND == 0)
                    states[half * kRows + row] = make_float2(m, l);
                bar_named(1, 2 * kRows);
                const float2 s0 = states[row], s1 = states[kRows + row];
                wait(o_full, n_b[0] - 1);
                if (n > 1)
                    wait(o_full + 8, n_b[1] - 1);
                tc_fence_after();
                m = fmaxf(s0.x, s1.x);
                const float f0 = s0.x == -INFINITY ? 0.f : fast_exp2(s0.x - m);
                const float f1 = s1.x == -INFINITY ? 0.f : fast_exp2(s1.x - m);
                l = fmaf(f0, s0.y, f1 * s1.y);
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
                for (int c = half * (D / 2); !dead && c < (half + 1) * (D / 2); c += 32) {
                    float o[32];
                    tmem_ld32(lanes + 256 + c, o);
                    tmem_wait_ld();
                    tmem_landed<32>(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] *= f0;
                    if (n > 1) { // (else the second buffer holds nothing)
                        float o1[32];
                        tmem_ld32(lanes + 384 + c, o1);
                        tmem_wait_ld();
                        tmem_landed<32>(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = fmaf(f1, o1[e], o[e]);
                    }
                    emit(c, o, inv);
                }
            }
            if (live && !g.whole && (two || half == 0))
                reinterpret_cast<float2 *>(rec + D * kUnitRows)[r] = make_float2(m, l);
            tc_fence_before(); // (the next p_full orders these reads before the next products)
            if (!two)
                bar_named(1, 2 * kRows); // each buffer's outputs were read by both
            if (g.whole)
                continue;
            // ---- a cut unit: the last CTA to arrive merges its records
            bar_named(1, 2 * kRows);
            const int64_t c_first = plan_owner(g.first_v, total, G);
            const int64_t last_v = g.first_v + (int64_t)(walk.s.tiles - 1) * g.weight;
            const int nseg = (int)(plan_owner(last_v, total, G) - c_first + 1);
            if (tid == 0) {
                const int last = atomic_add_acq_rel_gpu(p.counters + c_first, 1) == nseg - 1;
                if (last)
                    p.counters[c_first] = 0; // every arrival is in: ready for the next call
                misc[1] = last;
            }
            bar_named(1, 2 * kRows);
            if (!misc[1])
                continue;
            // (a CTA's records: 0 a unit it goes on with, 1 one that it begins)
            // thread: eight outputs of a row at a time, adjacent rows in adjacent threads; two
            // such pieces and up to two records are in flight together
            const float *first = record(c_first * 2 + 1), *rest = record((c_first + 1) * 2);
            const int pieces = g.rows * (D / 8);
            for (int i0 = tid; i0 < pieces; i0 += 4 * kRows) {
                MergeState st[2];
                int rr[2], d8[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = min(i0 + e * 2 * kRows, pieces - 1);
                    d8[e] = i / g.rows;
                    rr[e] = i - d8[e] * g.rows;
                    st[e].clear();
                }
                for (int q = 0; q < nseg; q += 2) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float *r0 = q == 0 ? first : rest + (int64_t)(q - 1) * 2 * RECORD;
                        const float *r1 = q + 1 < nseg ? rest + (int64_t)q * 2 * RECORD : nullptr;
                        st[e].template fold<D>(r0, r1, rr[e], d8[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float L = st[e].l, inv = L > 0.f || L != L ? 1.f / L : 0.f;
                    const float *o = st[e].o;
                    const int64_t pr = g.row0 + rr[e];
                    *reinterpret_cast<uint4 *>(
                        p.out +
                        ((walk.s.q0 + (pr >> p.log2_g)) * n_h + (g.kvh << p.log2_g) +
                         (pr & g_mask)) * D + 8 * d8[e]) =
                        make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv),
                                   pack_bf16x2(o[2] * inv, o[3] * inv),
                                   pack_bf16x2(o[4] * inv, o[5] * inv),
                                   pack_bf16x2(o[6] * inv, o[7] * inv));
                }
            }
        }
    } else {
        if constexpr (KIND != 0)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == kMmaWarp) {
            // ======================================================== matrix instructions
            // One thread runs the whole loop: a warp would pay a vote and a broadcast at each
            // of its waits and operands, which come one after another. The buffers take strict
            // turns (P V, then the next scores, of one, then of the other), which keeps one
            // in its softmax while the other has the tensor cores; with a thread per buffer
            // they fall into step and both wait for both.
            if (elect_one()) {
                constexpr uint32_t iS = tc_idesc_bf16(kRows, kRows, false);
                constexpr uint32_t iO = tc_idesc_bf16(kRows, D, true);
                constexpr uint64_t kHigh = tc_desc_high();
                constexpr uint32_t kSlotDesc = TILE >> 4;
                const uint32_t q_desc = (uint32_t)tc_desc(sbase, 16);
                const uint32_t k_ring = (uint32_t)tc_desc(ring, 16);
                const uint32_t v_ring = (uint32_t)tc_desc(ring, COL);
                uint32_t n_q = 0;             // segments
                uint32_t slot = 0, phase = 0; // ring position
                uint32_t np = 0, used = 0;    // per buffer: parity of its products with V; any yet
                auto ready = [&](uint32_t bar, uint32_t parity) {
                    if (!dead && !mbar_ready(bar, parity & 1u)) {
                        dead = true;
                        flag_error(p.dev_status, PA_DEV_TIMEOUT_BIT);
                    }
                    return !dead;
                };
                // the next ring slot, once it is filled
                auto take = [&](uint32_t &at) {
                    at = slot;
                    const uint32_t parity = phase;
                    if (++slot == SLOTS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                    return ready(kv_full + 8 * at, parity);
                };
                // output (+)= P V over 64 keys: both parts of the weights with one V tile
                auto products = [&](uint32_t tO, uint32_t tP, uint64_t v_desc, uint32_t more) {
#pragma unroll
                    for (int kk = 0; kk < kPart / 16; ++kk) {
                        tc_mma_ts(tO, tP + 8 * kk, v_desc + kk * (2048 >> 4), iO,
                                  kk > 0 ? 1 : more);
                        tc_mma_ts(tO, tP + kPart / 2 + 8 * kk, v_desc + kk * (2048 >> 4), iO, 1);
                    }
                };
                while (walk.next(g)) {
                    const int n = g.j1 - g.j0;
                    const bool two = g.halves == 2;
                    // Step k uses buffer k & 1: with two halves, half k & 1 and key tile k / 2;
                    // with one, key tile k. Products of step k, then scores of step k + 2.
                    const int steps = two ? 2 * n : n;
                    uint32_t ks = 0, v0 = 0, v1 = 0; // slots of the K tile and of the last V tiles
                    if (!ready(q_full, n_q))
                        break;
#pragma unroll 1
                    for (int k = -2; k < steps; ++k) {
                        const uint32_t b = k & 1;
                        const bool odd = b != 0, give = !two || odd; // a slot's last reader
                        if (k >= 0) { // output (+)= P V, in two parts
                            if (two ? !odd : k == n - 1) { // (else the scores' stage took it)
                                if (!take(v0))
                                    break;
                                v1 = v0;
                            }
                            const uint32_t vs = odd ? v1 : v0;
                            const uint64_t v_desc = kHigh | (v_ring + vs * kSlotDesc);
                            const uint32_t tO = 256 + b * 128, tS = b * 128;
                            const uint32_t more = k > 1;
                            if (!ready(p_full + 16 * b, np >> b))
                                break;
                            tc_fence_after();
                            products(tO, tS, v_desc, more);
                            tc_commit(a_full + 8 * b);
                            if (!ready(p_full + 16 * b + 8, np >> b))
                                break;
                            tc_fence_after();
                            products(tO, tS + kPart, v_desc + (kPart / 16) * (2048 >> 4), 1);
                            tc_commit(o_full + 8 * b);
                            if (give)
                                tc_commit(kv_empty + 8 * vs);
                            np ^= 1u << b;
                        }
                        if (k + 2 < steps) { // scores Q K^T of step k + 2
                            if (!two && k + 2 > 0 && !take(odd ? v0 : v1)) // V of step k + 1
                                break;
                            if (!(two && odd) && !take(ks))
                                break;
                            const uint64_t k_desc = kHigh | (k_ring + ks * kSlotDesc);
                            const uint64_t a_desc = kHigh | (q_desc + (two ? b * kSlotDesc : 0));
                            half_mask[b] = slot_mask[ks]; // (the softmax is done with the last one)
                            mbar_arrive(s_full + 8 * b);
                            // the buffer's last P V, which reads P where the scores go, must be done
                            if ((used >> b & 1u) && !ready(o_full + 8 * b, (np >> b) ^ 1u))
                                break;
                            used |= 1u << b;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk / 4) * COL + (kk % 4) * 32) >> 4;
                                tc_mma_ss(b * 128, a_desc + off, k_desc + off, iS, kk > 0);
                            }
                            tc_commit(s_full + 8 * b);
                            if (give)
                                tc_commit(kv_empty + 8 * ks);
                            if (k + 3 == steps)
                                tc_commit(q_empty);
                        }
                    }
                    if (dead)
                        break;
                    ++n_q;
                }
                if (dead) { // let what was issued finish (bounded) before the memory goes
                    tc_commit(drained);
                    mbar_poll(drained, 0);
                }
            }
            __syncwarp();
        } else if (warp == kCopyWarp) {
            // ============================================================== copies
            uint32_t n_q = 0, n_kv = 0;
            // ring of the copies: bf16 tiles, or tiles of codes
            constexpr int RING = KIND ? L::RAWS : SLOTS;
            const uint32_t full0 = KIND ? raw_full : kv_full, empty0 = KIND ? raw_empty : kv_empty;
            while (walk.next(g) && !dead) {
                const int nblk = (int)(((int64_t)walk.s.ctx + kBlockTokens - 1) / kBlockTokens);
                const int32_t *table = p.block_tables + (int64_t)walk.at.b * p.max_blocks;
                for (int j = g.j0; j < g.j1; ++j) {
                    // lanes 0-7 (and their copies): the tile's eight blocks
                    const int blk = j * kTileBlocks + (lane & 7);
                    const int32_t phys = blk < nblk ? __ldg(table + blk) : -1;
                    const bool ok = phys >= 0 && phys < p.num_blocks;
                    const uint32_t bad =
                        __ballot_sync(0xffffffffu, blk < nblk && !ok) & 0xffu;
                    if (bad && lane == 0)
                        flag_error(p.dev_status, PA_DEV_BAD_BLOCK_BIT);
                    const uint32_t have = __ballot_sync(0xffffffffu, ok) & 0xffu;
                    const int32_t prow = ok ? phys * p.n_kv + g.kvh : -1; // (block, head) tile
                    int32_t rows[kTileBlocks];
#pragma unroll
                    for (int i = 0; i < kTileBlocks; ++i)
                        rows[i] = __shfl_sync(0xffffffffu, prow, i);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++n_kv) {
                        const uint32_t slot = n_kv % RING;
                        if (!wait(empty0 + 8 * slot, n_kv / RING + 1))
                            break;
                        const uint32_t full = warp_uniform(full0 + 8 * slot);
                        if constexpr (KIND == 0) {
                            const CUtensorMap *tm = kv ? &tmV : &tmK;
                            const uint32_t dst = warp_uniform(ring + slot * TILE);
                            if (elect_one()) {
                                const uint64_t pol = l2_policy_evict_normal();
                                slot_mask[slot] = (int32_t)bad;
                                mbar_arrive_expect_tx(full, TILE);
                                // absent and bad blocks: a box outside the pool arrives as zeros
                                const int32_t outside =
                                    (int32_t)(p.num_blocks * p.n_kv * kBlockTokens);
#pragma unroll
                                for (int i = 0; i < kTileBlocks; ++i) {
                                    const int32_t y = rows[i] >= 0 ? rows[i] * kBlockTokens : outside;
#pragma unroll
                                    for (int c = 0; c < HALVES; ++c)
                                        tma_load_2d(dst + c * COL + i * 2048, tm, c * 64, y, full,
                                                    pol);
                                }
                            }
                        } else {
                            constexpr uint32_t BLOCK = kBlockTokens * L::ROWB;
                            const uint8_t *pool =
                                static_cast<const uint8_t *>(kv ? p.v_cache : p.k_cache);
                            const uint32_t dst = warp_uniform(sbase + L::kOffRaw + slot * L::RAW);
                            if (elect_one()) {
                                const uint64_t pol = l2_policy_evict_normal();
                                raw_mask[slot] = (int32_t)(have | bad << 8);
                                // the K tile brings the scales of both
                                mbar_arrive_expect_tx(full, __popc(have) * (BLOCK + (kv ? 0 : 128)));
#pragma unroll
                                for (int i = 0; i < kTileBlocks; ++i) {
                                    if (rows[i] < 0)
                                        continue;
                                    bulk_load_1d(dst + i * BLOCK, pool + (int64_t)rows[i] * BLOCK,
                                                 BLOCK, full, pol);
                                    if (kv == 0) {
                                        const int64_t at = (int64_t)rows[i] * kBlockTokens;
                                        const uint32_t sc = dst + kRows * L::ROWB + i * 64;
                                        bulk_load_1d(sc, p.k_scale + at, 64, full, pol);
                                        bulk_load_1d(sc + kRows * 4, p.v_scale + at, 64, full, pol);
                                    }
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if (dead)
                        break;
                    if (j == g.j0) { // the unit's queries, once the last unit's are read
                        if (!wait(q_empty, n_q + 1))
                            break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(q_full, (uint32_t)(g.halves * TILE));
                            const int32_t t0 = (int32_t)(walk.s.q0 + (g.row0 >> p.log2_g));
                            for (int i = 0; i < g.halves; ++i)
                                for (int c = 0; c < HALVES; ++c)
                                    tma_load_3d(sbase + i * TILE + c * COL, &tmQ, c * 64,
                                                g.kvh << p.log2_g, t0 + i * (kRows >> p.log2_g),
                                                q_full);
                        }
                        __syncwarp();
                        ++n_q;
                    }
                }
            }
            zero_rows(lane, 32);
            if (dead) { // copies in flight land (bounded) before the memory goes
                for (uint32_t n = n_kv > RING ? n_kv - RING : 0; n < n_kv; ++n)
                    mbar_poll(full0 + 8 * (n % RING), (n / RING) & 1u);
                if (n_q)
                    mbar_poll(q_full, (n_q - 1) & 1u);
            }
        } else if constexpr (KIND != 0) {
            // ======================================================= codes into bf16
            constexpr int CPR = L::ROWB / 16; // 16-byte chunks per row
            constexpr int CONV = kConvWarps * 32, STEP = CONV / CPR;
            static_assert(STEP % 8 == 0, "rows of one thread lie alike in the swizzle");
            const int t = tid - (kCopyWarp + 1) * 32;
            // where the thread's chunk of a row goes: 16-byte chunks of the row's bf16 values
            const int flip = KIND == 1 && CPR == 8 ? (t % CPR) >> 2 : 0;
            uint32_t at[4];
#pragma unroll
            for (int i = 0; i < (KIND == 1 ? 2 : 4); ++i) {
                const int oc = KIND == 1 ? 2 * (t % CPR) + (i ^ flip) : 4 * (t % CPR) + i;
                at[i] = (oc / 8) * COL + (((oc % 8) ^ (t / CPR & 7)) << 4);
            }
            uint32_t n_kv = 0, n_tile = 0;
            while (walk.next(g) && !dead) {
                for (int j = g.j0; j < g.j1 && !dead; ++j, ++n_tile) {
                    const int valid = min(walk.s.ctx - j * kRows, kRows);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++n_kv) {
                        const uint32_t from = n_kv % L::RAWS, slot = n_kv % SLOTS;
                        if (!wait(raw_full + 8 * from, n_kv / L::RAWS) ||
                            !wait(kv_empty + 8 * slot, n_kv / SLOTS + 1))
                            break;
                        const uint32_t dst = ring + slot * TILE;
                        const uint8_t *raw = smem + L::kOffRaw + from * L::RAW;
                        const int mask = raw_mask[from];
                        // rows of absent and bad blocks and behind the context are zero
                        auto present = [&](int r) {
                            return r < valid && ((mask >> (r / kBlockTokens)) & 1);
                        };
                        if (t == 0)
                            slot_mask[slot] = mask >> 8;
                        if (kv == 0 && t < kRows) {
                            const float *in =
                                reinterpret_cast<const float *>(raw + kRows * L::ROWB);
                            float *sc = reinterpret_cast<float *>(smem + L::kOffScales) +
                                        (n_tile % kScaleRing) * 2 * kRows;
                            sc[t] = present(t) ? in[t] * p.scale_log2 : 0.f;
                            sc[kRows + t] = present(t) ? in[kRows + t] : 0.f;
                        }
                        // Chunk t + i * CONV of the tile: its row moves by STEP, a multiple of the
                        // swizzle's eight, so the addresses move by constants.
                        uint32_t in = smem_u32(raw) + 16 * t, out = dst + t / CPR * 128;
#pragma unroll 1 // (unrolled, its instructions push the other warps' out of the cache)
                        for (int r = t / CPR; r < kRows; r += STEP) {
                            uint32_t w[4];
                            lds128(in, w);
                            // rows that are not there are zero (INT4: 8 is code 0)
                            if (!present(r))
                                w[0] = w[1] = w[2] = w[3] = 0;
                            if constexpr (KIND == 1) {
                                // (a row's second 64 columns take its chunks in the other
                                // order: a row's eight threads then write to different banks)
                                const uint32_t a0 = flip ? w[2] : w[0], a1 = flip ? w[3] : w[1];
                                const uint32_t b0 = flip ? w[0] : w[2], b1 = flip ? w[1] : w[3];
                                sts128(out + at[0], code8_bf2<0x4140>(a0), code8_bf2<0x4342>(a0),
                                       code8_bf2<0x4140>(a1), code8_bf2<0x4342>(a1));
                                sts128(out + at[1], code8_bf2<0x4140>(b0), code8_bf2<0x4342>(b0),
                                       code8_bf2<0x4140>(b1), code8_bf2<0x4342>(b1));
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t a = w[i] ^ 0x88888888u, b = a >> 4;
                                    sts128(out + at[i], code4_bf2<0>(a, b), code4_bf2<1>(a, b),
                                           code4_bf2<2>(a, b), code4_bf2<3>(a, b));
                                }
                            }
                            in += 16 * CONV;
                            out += STEP * 128;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(kv_full + 8 * slot);
                            mbar_arrive(raw_empty + 8 * from);
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, 512);
}

template <int D, int KIND>
cudaError_t launch_of(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                      const CrossParams &p, cudaStream_t stream)
{
    constexpr int bytes = Smem<D, KIND>::kBytes;
    static_assert(bytes <= 232448 && bytes > 116 * 1024, "one CTA per SM");
    static std::atomic<bool> raised[kRaisedDevices]; // the opt-in to that much, once per device
    const cudaError_t e =
        raise_shared_memory(raised, reinterpret_cast<const void *>(cross_kernel<D, KIND>), bytes);
    if (e != cudaSuccess)
        return e;
    cross_kernel<D, KIND><<<p.num_ctas, Smem<D, KIND>::kThreads, bytes, stream>>>(tq, tk, tv, p);
    return cudaGetLastError();
}

size_t counter_bytes(int num_ctas) { return ((size_t)num_ctas * 4 + 255) / 256 * 256; }

} // namespace

size_t cross_workspace_bytes(int d_h, int num_ctas)
{
    return counter_bytes(num_ctas) + (size_t)num_ctas * 2 * record_floats(d_h) * sizeof(float);
}

cudaError_t launch_cross(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                         const CrossArgs &a, cudaStream_t stream)
{
    CrossParams p;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.cu_q = a.cu_q;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.counters = static_cast<int32_t *>(a.workspace);
    p.records = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) +
                                          counter_bytes(a.num_ctas));
    p.dev_status = a.dev_status;
    p.num_q = a.num_q;
    p.num_blocks = a.num_blocks;
    p.num_seqs = a.num_seqs;
    p.n_kv = a.n_kv;
    p.log2_g = a.g == 1 ? 0 : a.g == 2 ? 1 : a.g == 4 ? 2 : a.g == 8 ? 3 : 4;
    p.max_blocks = a.max_blocks;
    p.num_ctas = a.num_ctas;
    p.scale_log2 = a.scale_log2;
    const int kind = a.kind;
    if (a.d_h == 128)
        return kind == 0   ? launch_of<128, 0>(tq, tk, tv, p, stream)
               : kind == 1 ? launch_of<128, 1>(tq, tk, tv, p, stream)
                           : launch_of<128, 2>(tq, tk, tv, p, stream);
    return kind == 0   ? launch_of<64, 0>(tq, tk, tv, p, stream)
           : kind == 1 ? launch_of<64, 1>(tq, tk, tv, p, stream)
                       : launch_of<64, 2>(tq, tk, tv, p, stream);
}

} // namespace pa
