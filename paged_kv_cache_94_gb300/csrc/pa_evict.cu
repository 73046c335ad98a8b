// Eviction from a paged cache by accumulated attention weight.
//
// select_kernel: which tokens of each (sequence, kv head) stay. With n = ctx_b,
//   k = min(n, budget), r = min(recent, k): tokens n - r .. n - 1, and of the
//   m = n - r before them the k - r of largest mass, ties to the lowest index,
//   in ascending order. The k - r th largest key (masses as unsigned integers
//   in their order) is found from counts over 2048 bins of the keys' range in
//   shared memory, again over the bin that holds it while many do, then by
//   comparing the few keys of its bin with each other; one more sweep counts what
//   lies above it and writes the indices at their ranks. Ranks come from warp
//   ballots and prefix sums, so the result does not depend on any order of
//   execution.
//   A row is 4 n bytes, read once: latency-bound. So a long row is cut over a
//   cluster of up to 8 CTAs (counts joined in the first one's shared memory) and
//   the keys stay in shared memory between the sweeps; rows too long for that, by the
//   stride of the masses, read them again from L2. 512 rows of 900..4096 tokens: 17 us a
//   call (14 on the GPU, in two waves; 16 with a stride of 131072), 32 of 32K..128K: 31 us
//   (11 and 40 thousand cycles a CTA: loads, then six steps of which each is one or two
//   barriers).
//
// compact_kernel: row i of the new block table = row keep[i] of the old one,
//   for K, V, their scales and the masses. Bound by HBM: each kept row is read
//   and written once. A CTA moves 1024 16-byte pieces of K and as many of V:
//   64 bf16 rows of 128, more of narrower ones. The rows' places are looked up
//   once into shared memory; then every thread has eight 16-byte loads in
//   flight before its first store. 64 x 8 x 1024 bf16 rows of 128: 88.5 us, 6120
//   GB/s, 0.91 of the measured copy rate; INT8 rows of 4 x 8 x 16384: 59.5 us, 0.71,
//   each scattered scale costing a 32-byte sector.
#include <cooperative_groups.h>

#include "pa_internal.h"
#include "pa_launch.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeys = 48; // keys of a thread kept in shared memory (up to 47: two CTAs per SM)

// Masses as unsigned integers of the same order. -0 equals +0; NaN lies below
// everything, so a token whose mass is not a number goes first.
constexpr uint32_t kZeroKey = 0x80000000u;
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f); // -0 + 0 = +0
    if (x != x)
        return 0u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kFew = 512; // candidates that are ranked by comparing them with each other

struct SelShared {
    int32_t hist[kBins];
    int32_t total[kBins]; // the cluster's counts (first CTA)
    uint32_t few[kFew];   // the candidates' keys (first CTA)
    int32_t n_few;
    int32_t warp_sum[kSelWarps];
    uint32_t low[kSelWarps], low_pos[kSelWarps], high[kSelWarps]; // least keys, greatest
    uint32_t lo, hi;      // result of a step: the threshold's range,
    int32_t need, left;   // its rank there, keys there
    int32_t gt[kSelWarps], eq[kSelWarps];
    int32_t cta_gt, cta_eq;
};

// CACHED: the keys stay in shared memory (each thread's own). CLUSTER: several CTAs per row.
// Three CTAs per SM where a CTA has a row to itself (many rows: 16.9 us against 18.4 with two),
// two in a cluster (few rows; with three its registers spill, 32.8 us against 31.4).
template <bool CACHED, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, CLUSTER ? 2 : 3)
select_kernel(const float *__restrict__ mass, int64_t stride,
              const int32_t *__restrict__ context_lens, int n_kv, int budget, int recent,
              int32_t *__restrict__ keep, int32_t *__restrict__ keep_lens, int32_t *dev_status)
{
    __shared__ SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = CLUSTER ? (int)cluster.num_blocks() : 1;
    const int rank = CLUSTER ? (int)cluster.block_rank() : 0;
    auto sync = [&]() {
        if constexpr (CLUSTER)
            cluster.sync();
        else
            __syncthreads();
    };
    auto of = [&](int q) { return CLUSTER ? cluster.map_shared_rank(&sh, q) : &sh; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t u = blockIdx.x / C; // b * n_kv + kv head
    const int b = (int)(u / n_kv);
    int32_t n = __ldg(context_lens + b);
    if (n < 0 || n > stride) {
        if (tid == 0 && dev_status)
            atomicOr(dev_status, PA_DEV_BAD_CONTEXT_BIT);
        n = 0;
    }
    const int32_t k = min(n, budget), r = min(recent, k);
    const int32_t m = n - r, want = k - r; // choose `want` of tokens [0, m)
    int32_t *out = keep + u * budget;

    // what needs no choice: the recent tokens, the unused tail, the count
    // (64-bit indices: one step beyond a budget near 2^31 passes 32)
    for (int64_t i = (int64_t)want + rank * kSelThreads + tid; i < budget; i += C * kSelThreads)
        out[i] = i < k ? m + (int32_t)(i - want) : -1;
    if (tid == 0 && rank == 0 && u % n_kv == 0)
        keep_lens[b] = k;
    if (want == m) { // nothing to evict (the same in every CTA of the cluster)
        for (int64_t i = rank * kSelThreads + tid; i < want; i += C * kSelThreads)
            out[i] = (int32_t)i;
        return;
    }
    if (want == 0)
        return;

    // this warp's run of tokens: whole rounds of 32
    const int32_t warps = C * kSelWarps;
    const int32_t rounds = (int32_t)(((int64_t)m + 32 * warps - 1) / (32 * warps));
    const int64_t first = (int64_t)(rank * kSelWarps + warp) * rounds * 32 + lane;
    const float *row = mass + u * stride;
    auto load = [&](int it) -> uint32_t { // (only called for tokens below m)
        return key_of(__ldg(row + first + (int64_t)it * 32));
    };
    extern __shared__ uint32_t keys[];
    uint32_t *mine = keys + warp * rounds * 32 + lane;
    if constexpr (CACHED) {
#pragma unroll 8
        for (int it = 0; it < rounds; ++it)
            mine[it * 32] = first + it * 32 < m ? load(it) : 0u;
    }
    // f(round, key, valid) over this thread's tokens, all lanes of a warp together
    auto sweep = [&](auto f) {
#pragma unroll 4
        for (int it = 0; it < rounds; ++it) {
            const bool in = first + (int64_t)it * 32 < m;
            f(it, CACHED ? mine[it * 32] : in ? load(it) : 0u, in);
        }
    };

    // The range of the keys: all, and of the masses above zero.
    uint32_t lowest = 0xffffffffu, low_pos = 0xffffffffu, hi = 0;
    sweep([&](int, uint32_t key, bool in) {
        if (in) {
            lowest = min(lowest, key);
            low_pos = key > kZeroKey ? min(low_pos, key) : low_pos;
            hi = max(hi, key);
        }
    });
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    low_pos = __reduce_min_sync(0xffffffffu, low_pos);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.low[warp] = lowest;
        sh.low_pos[warp] = low_pos;
        sh.high[warp] = hi;
    }
    if (tid == 0)
        sh.n_few = 0;
    for (int i = tid; i < kBins; i += kSelThreads)
        sh.hist[i] = sh.total[i] = 0;
    sync();
    for (int i = lane; i < C * kSelWarps; i += 32) { // every warp joins all of the row's
        SelShared *s = of(i / kSelWarps);
        lowest = min(lowest, s->low[i % kSelWarps]);
        low_pos = min(low_pos, s->low_pos[i % kSelWarps]);
        hi = max(hi, s->high[i % kSelWarps]);
    }
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    low_pos = __reduce_min_sync(0xffffffffu, low_pos);
    hi = __reduce_max_sync(0xffffffffu, hi);

    // The `want`-th largest key lies in [lo, hi] and is the need-th largest of the `left`
    // keys there. Counts over up to 2048 equal bins of that range narrow it, first of the
    // masses above zero (zeros would stretch the range over all the exponents), until few are
    // left, which are compared with each other.
    uint32_t lo = low_pos <= hi && m > kFew ? low_pos : lowest;
    int32_t need = want, left = m;
    bool clean = true; // the counts are zero
#pragma unroll 1
    while (left > kFew && (lo < hi || (clean && lo > lowest))) {
        const int bits = 32 - __clz(hi - lo), shift = max(0, bits - 11);
        if (!clean) {
            for (int i = tid; i < kBins; i += kSelThreads) {
                sh.hist[i] = 0;
                if (CLUSTER)
                    sh.total[i] = 0;
            }
            sync(); // (the first CTA's totals are zero before anyone adds to them)
        }
        clean = false;
        sweep([&](int, uint32_t key, bool in) {
            if (in && key - lo <= hi - lo)
                atomicAdd(&sh.hist[(key - lo) >> shift], 1);
        });
        __syncthreads();
        if constexpr (CLUSTER) {
            int32_t *total = of(0)->total;
            for (int i = tid; i < kBins; i += kSelThreads)
                if (sh.hist[i])
                    atomicAdd(total + i, sh.hist[i]);
            cluster.sync();
        }
        if (rank == 0) { // the bin: counts from the top until `need` are covered
            const int32_t *t = CLUSTER ? sh.total : sh.hist;
            constexpr int PER = kBins / kSelThreads;
            int32_t c[PER], sum = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                c[j] = t[kBins - 1 - (tid * PER + j)];
                sum += c[j];
            }
            int32_t x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o)
                    x += y;
            }
            if (lane == 31)
                sh.warp_sum[warp] = x;
            __syncthreads();
            int32_t before = x - sum;
#pragma unroll
            for (int w = 0; w < kSelWarps; ++w)
                before += w < warp ? sh.warp_sum[w] : 0;
            const bool here = before < need && need <= before + sum; // in one thread at most
            const bool below = tid == kSelThreads - 1 && before + sum < need;
            if (here || below) { // `below`: among the masses that are not above zero
                uint32_t new_lo = lowest, new_hi = lo - 1;
                int32_t new_left = m - (before + sum), new_need = need - (before + sum);
                if (here) {
                    int j = 0;
                    while (before + c[j] < need)
                        before += c[j++];
                    new_lo = lo + ((uint32_t)(kBins - 1 - (tid * PER + j)) << shift);
                    new_hi = min(hi, new_lo + ((1u << shift) - 1));
                    new_left = c[j];
                    new_need = need - before;
                }
                for (int q = 0; q < C; ++q) {
                    SelShared *s = of(q);
                    s->lo = new_lo;
                    s->hi = new_hi;
                    s->need = new_need;
                    s->left = new_left;
                }
            }
        }
        sync();
        lo = sh.lo;
        hi = sh.hi;
        need = sh.need;
        left = sh.left;
    }
    if (lo < hi) { // few: the need-th largest of them by comparing all with all
        SelShared *to = of(0);
        sweep([&](int, uint32_t key, bool in) {
            if (in && key - lo <= hi - lo)
                to->few[atomicAdd(&to->n_few, 1)] = key;
        });
        sync();
        if (rank == 0 && tid < left) {
            const uint32_t own = sh.few[tid];
            int32_t above = 0, same = 0;
            for (int i = 0; i < left; ++i) {
                above += sh.few[i] > own;
                same += sh.few[i] == own;
            }
            if (above < need && need <= above + same) // one key (every thread that has it)
                for (int q = 0; q < C; ++q) {
                    of(q)->lo = own;
                    of(q)->need = need - above;
                }
        }
        sync();
        lo = sh.lo;
        need = sh.need;
    }
    const uint32_t threshold = lo;

    // ranks: tokens above the threshold, and the first `need` of those equal to it
    int32_t gt = 0, eq = 0;
    sweep([&](int, uint32_t key, bool in) {
        gt += in && key > threshold;
        eq += in && key == threshold;
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sh.gt[warp] = gt;
        sh.eq[warp] = eq;
    }
    __syncthreads();
    int32_t gt0 = 0, eq0 = 0; // before this warp
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        gt0 += w < warp ? sh.gt[w] : 0;
        eq0 += w < warp ? sh.eq[w] : 0;
    }
    if constexpr (CLUSTER) {
        if (tid == 0) {
            int32_t g = 0, e = 0;
            for (int w = 0; w < kSelWarps; ++w) {
                g += sh.gt[w];
                e += sh.eq[w];
            }
            sh.cta_gt = g;
            sh.cta_eq = e;
        }
        cluster.sync();
        for (int q = 0; q < rank; ++q) {
            gt0 += of(q)->cta_gt;
            eq0 += of(q)->cta_eq;
        }
    }
    const uint32_t below = (1u << lane) - 1;
    sweep([&](int it, uint32_t key, bool in) {
        const uint32_t g = __ballot_sync(0xffffffffu, in && key > threshold);
        const uint32_t e = __ballot_sync(0xffffffffu, in && key == threshold);
        const int32_t gb = gt0 + __popc(g & below), eb = eq0 + __popc(e & below);
        if (in && (key > threshold || (key == threshold && eb < need)))
            out[gb + min(eb, need)] = (int32_t)(first + (int64_t)it * 32);
        gt0 += __popc(g);
        eq0 += __popc(e);
    });
    if constexpr (CLUSTER)
        cluster.sync(); // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------------------
constexpr int kCompThreads = 256;
constexpr int kPieces = 1024;                             // 16-byte pieces of K (and of V) per CTA
constexpr int kPerThread = 2 * kPieces / kCompThreads;    // 8

// PPR: 16-byte pieces per row
template <int PPR>
__global__ void __launch_bounds__(kCompThreads)
compact_kernel(uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
               const int32_t *__restrict__ tables, int max_blocks,
               const int32_t *__restrict__ keep, int budget, const int32_t *__restrict__ keep_lens,
               const int32_t *__restrict__ new_tables, int new_blocks,
               const float *__restrict__ mass, float *mass_out, int64_t num_blocks, int n_kv,
               int tiles, int32_t *dev_status)
{
    constexpr int ROWS = kPieces / PPR;
    __shared__ int32_t src[ROWS], dst[ROWS]; // pool rows; -1: not moved
    const int64_t u = blockIdx.x / tiles;    // b * n_kv + kv head
    const int b = (int)(u / n_kv), h = (int)(u - (int64_t)b * n_kv);
    const int32_t row0 = (int32_t)(blockIdx.x - u * tiles) * ROWS;
    const int64_t old_cap = (int64_t)max_blocks * 16, new_cap = (int64_t)new_blocks * 16;
    int32_t kept = __ldg(keep_lens + b);
    if (kept < 0 || kept > budget || kept > new_cap) {
        if (threadIdx.x == 0 && dev_status)
            atomicOr(dev_status, PA_DEV_BAD_CONTEXT_BIT);
        kept = 0;
    }
    for (int t = threadIdx.x; t < ROWS; t += kCompThreads) {
        const int32_t i = row0 + t;
        int32_t s = -1, d = -1;
        float w = 0.f;
        if (i < kept) {
            const int32_t j = __ldg(keep + u * budget + i);
            if (j < 0 || j >= old_cap) {
                if (dev_status)
                    atomicOr(dev_status, PA_DEV_BAD_CONTEXT_BIT);
            } else {
                const int32_t sb = __ldg(tables + (int64_t)b * max_blocks + j / 16);
                const int32_t db = __ldg(new_tables + (int64_t)b * new_blocks + i / 16);
                if (sb < 0 || sb >= num_blocks || db < 0 || db >= num_blocks) {
                    if (dev_status)
                        atomicOr(dev_status, PA_DEV_BAD_BLOCK_BIT);
                } else {
                    s = (sb * n_kv + h) * 16 + j % 16;
                    d = (db * n_kv + h) * 16 + i % 16;
                    if (k_scale) {
                        k_scale[d] = k_scale[s];
                        v_scale[d] = v_scale[s];
                    }
                    if (mass)
                        w = __ldg(mass + u * old_cap + j);
                }
            }
        }
        src[t] = s;
        dst[t] = d;
        if (mass_out && i < new_cap)
            mass_out[u * new_cap + i] = w;
    }
    if (row0 >= kept)
        return;
    __syncthreads();
    uint4 x[kPerThread];
    // piece c of the CTA's 2 * kPieces: row c / (2 PPR), then K's pieces, then V's
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
        const int c = e * kCompThreads + threadIdx.x, t = c / (2 * PPR), o = c % (2 * PPR);
        const uint8_t *pool = o < PPR ? k_cache : v_cache;
        if (src[t] >= 0)
            x[e] = __ldcs(reinterpret_cast<const uint4 *>(pool) + (int64_t)src[t] * PPR + o % PPR);
    }
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
        const int c = e * kCompThreads + threadIdx.x, t = c / (2 * PPR), o = c % (2 * PPR);
        uint8_t *pool = o < PPR ? k_cache : v_cache;
        if (src[t] >= 0)
            reinterpret_cast<uint4 *>(pool)[(int64_t)dst[t] * PPR + o % PPR] = x[e];
    }
}

} // namespace

cudaError_t launch_evict_select(const float *mass, int64_t stride, const int32_t *context_lens,
                                int num_seqs, int n_kv, int budget, int recent, int32_t *keep,
                                int32_t *keep_lens, int sms, int32_t *dev_status,
                                cudaStream_t stream)
{
    const int64_t rows = (int64_t)num_seqs * n_kv;
    // CTAs per row: more while the rows leave SMs idle and each CTA still has
    // eight keys per thread
    int C = 1;
    while (C < 8 && rows * C < 2 * sms && stride / C > 8 * kSelThreads)
        C *= 2;
    if (rows * C > INT32_MAX)
        return cudaErrorInvalidValue;
    const int64_t per_thread = (stride + (int64_t)C * kSelThreads - 1) / ((int64_t)C * kSelThreads);
    const bool cached = per_thread <= kKeys;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    auto kernel = C > 1 ? cached ? select_kernel<true, true> : select_kernel<false, true>
                        : cached ? select_kernel<true, false> : select_kernel<false, false>;
    if (cached)
        cfg.dynamicSmemBytes = (size_t)per_thread * kSelThreads * sizeof(uint32_t);
    if (cfg.dynamicSmemBytes > 16 * 1024) { // (with the static part, over the 48 KiB default at most)
        static std::atomic<bool> raised[2][kRaisedDevices]; // per kernel that keeps its keys
        const cudaError_t e =
            raise_shared_memory(raised[C > 1], reinterpret_cast<const void *>(kernel),
                                kKeys * kSelThreads * (int)sizeof(uint32_t));
        if (e != cudaSuccess)
            return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, mass, stride, context_lens, n_kv, budget, recent, keep,
                              keep_lens, dev_status);
}

cudaError_t launch_evict_compact(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                                 const int32_t *tables, int max_blocks, const int32_t *keep,
                                 int budget, const int32_t *keep_lens, const int32_t *new_tables,
                                 int new_blocks, const float *mass, float *mass_out, int num_seqs,
                                 int64_t num_blocks, int n_kv, int row_bytes, int32_t *dev_status,
                                 cudaStream_t stream)
{
    const int ppr = row_bytes / 16;
    const int rows = kPieces / ppr;
    // without masses only rows to move; with them the entries behind those are zeroed
    const int64_t new_cap = (int64_t)new_blocks * 16;
    const int64_t cover = mass_out || new_cap < budget ? new_cap : budget;
    const int64_t tiles = (cover + rows - 1) / rows;
    const int64_t grid = (int64_t)num_seqs * n_kv * tiles;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)grid, kCompThreads, 0, stream>>>(
            static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), k_scale, v_scale,
            tables, max_blocks, keep, budget, keep_lens, new_tables, new_blocks, mass, mass_out,
            num_blocks, n_kv, (int)tiles, dev_status);
        return cudaGetLastError();
    };
    switch (ppr) {
    case 16: return go(compact_kernel<16>);
    case 8: return go(compact_kernel<8>);
    case 4: return go(compact_kernel<4>);
    case 2: return go(compact_kernel<2>);
    default: return cudaErrorInvalidValue;
    }
}

} // namespace pa
