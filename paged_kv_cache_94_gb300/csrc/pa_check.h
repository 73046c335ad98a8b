// Which of the two checking warps of window attention takes the V tile of a CTA's key tile n
// (pa_cross_kernel.cuh, kCheck), shared by host and device code.
//
// K and V tiles take the ring's slots in turn, so V tile n stands in slot (2 n + 1) % slots, and
// where four divides the number of slots all tiles of a slot go to one warp. A slot is filled
// again only after the products of its tile, which wait for that warp's arrival: the barrier of
// what has landed is never two phases ahead of the warp that waits on it, and its parity never
// mistaken. (Tiles dealt out one by one, with both warps waiting for each, let the other warp's
// tiles run ahead of one that had not polled yet.)
#pragma once

#include "pa_plan.h"

namespace pa {

PA_HD constexpr uint32_t check_slot(uint32_t n_tile, uint32_t slots)
{
    return (2 * n_tile + 1) % slots;
}

PA_HD constexpr uint32_t check_warp(uint32_t n_tile) { return n_tile & 1; }

} // namespace pa
