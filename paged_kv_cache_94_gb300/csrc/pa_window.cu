// Compiled kernels of causal attention within a sliding window and to a sequence's first
// tokens (pa_cross_kernel.cuh with its mask, WIN).
//
//     token i of sequence b's n: position p = ctx_b - n + i; sees j <= p with j > p - window or
//     j < n_first;  out = sum_j softmax(scale <q, K_j>)_j V_j over those
//
// What bounds it: 4 d_h FLOP per (query row, key it sees) against each row of K and V once per
// (kv head, 256 query rows). Prompts are bound by the tensor cores, whose products with V count
// twice (weights in two bf16 parts); short windows and drafts by the chain of a tile.
//
// Which tiles. A unit (256 / g tokens of a kv head) sees the blocks of the first tokens and those
// from its first token's window to its last token; its tiles are eight of these blocks each, from
// wherever they begin, so that a window costs its own length and 4 first tokens one block, not a
// tile each. The number of tiles in front of a unit is a closed sum (tiles_before), by which the
// line is cut as evenly as cross attention's.
//
// The mask. Only tiles with a key that some row does not see take it: 64 bits a row from three
// shifts, a select a score. In the same tiles V entries that are not finite are taken out before
// the products (two warps that bf16 pools leave idle), since 0 times NaN is NaN, and put NaN into
// the rows that see them. A row whose seen scores are all minus infinity has a base of its own
// (kNoWeight) and comes out as NaN; one that sees nothing, as zeros.
//
// Measured on a GB300 (g = 4, d_h 128, bf16 unless said): one prompt of 16384 tokens
// 2020..2200 us as the power cap has it, 1000..1090 TFLOP/s with each product counted once: with
// those for both parts of the weights 1500..1630, 0.87..0.95 of what the cap sustains (1726).
// Eight chunks of 512..2048 tokens over 2048..8192 with a window of 4096: 650..705 us, 900..975
// TFLOP/s. 48 drafts of 1..8 tokens over 200..8192: 119 us, 5210 GB/s, 0.77 of the measured copy
// rate. 24 prompts of 33..1999 tokens, 16 heads of 64, g = 1, a window of 333: 146..151 us, where
// nearly every tile is masked and a unit has five. INT8, 16..256 tokens over 512..8192, g = 1, a
// window of 2000: 260 us (INT4 251) with the issue slots 51% busy; of a warp's time 37% is waits for
// tensor memory and for codes, 14% fixed latencies, 9% instruction fetch. Its loops are sensitive
// to their size all the same: weights and codes in fp16, a quarter fewer instructions but two
// loops more, took 279, a mask formed key by key instead of by words 315.
#include "pa_cross_kernel.cuh"

namespace pa {

cudaError_t launch_window(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const CrossArgs &a, cudaStream_t stream)
{
    return launch_any<1>(tq, tk, tv, a, stream);
}

} // namespace pa
