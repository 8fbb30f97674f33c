// piece_ring.h -- how the warps of a CTA hand pieces of work on, where any wait may
// give up. One warp puts pieces, the others take them; piece n lies in place n & 1
// until every taker has given it back. No CUDA here but the qualifier: the CPU tests
// run the same code with threads for warps.
//
// A wait says whether its barrier's phase has completed, the same to all lanes of a
// warp. One that gave up has seen nothing: a taker then leaves without a look at the
// place (an earlier piece may lie there, or none), and the putter writes no more (the
// place may be in use). Takers that left give nothing back, so the putter's wait gives
// up in turn, and then those of the others: all of them end.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_PIECE __device__ __forceinline__
#else
#define MOE_PIECE inline
#endif

namespace moe {

// Whether piece `number` is there to be worked on. wait_full(place, parity);
// is_end(place): no piece, the work is done.
template <class Wait, class IsEnd>
MOE_PIECE bool take_piece(int number, Wait wait_full, IsEnd is_end) {
    return wait_full(number & 1, (uint32_t)(number >> 1) & 1u) && !is_end(number & 1);
}

// Writes piece `number`, once the one before it in its place has been given back.
// wait_empty(place, parity), write(place). False: nothing was written, and no piece
// may follow.
template <class Wait, class Write>
MOE_PIECE bool put_piece(int number, Wait wait_empty, Write write) {
    if (!wait_empty(number & 1, ((uint32_t)(number >> 1) & 1u) ^ 1u)) return false;
    write(number & 1);
    return true;
}

// Whether one of four warps says yes to question `number` (they ask the same ones in
// turn). A barrier of the hardware would wait for a warp that has left; here
// arrive(), by one lane of each, and wait(parity) are of an mbarrier of four arrivals.
// Votes lie in two places by turns: a warp votes on the next but one only after all
// have voted on the next, and so have read this one.
struct Votes {
    uint8_t yes[2][4];
};
template <class Arrive, class Wait>
MOE_PIECE bool any_of_four(Votes& votes, int number, int warp, bool mine, Arrive arrive, Wait wait) {
    volatile uint8_t* yes = votes.yes[number & 1];
    arrive([&] { yes[warp] = mine; });
    wait((uint32_t)number & 1u);
    return yes[0] | yes[1] | yes[2] | yes[3];
}

}  // namespace moe
