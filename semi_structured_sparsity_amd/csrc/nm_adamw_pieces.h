// How the tensors of an optimiser step are spread over launches (host code without HIP).
#pragma once

#include <stdint.h>

namespace nm {

// A launch's work items (blocks x threads) are counted in 32 bits: blocks of 256 threads below 2^24.
constexpr int64_t kAdamWMostBlocks = (1 << 24) - 1;

// Calls add(i, at, n, block) for the pieces of the tensors of size(i) elements in order, each piece
// elements at .. at + n - 1 of tensor i and the launch's blocks from block on (chunk elements each), and
// flush() after the last piece of a launch.  A launch holds at most max_pieces pieces and most blocks; a
// tensor that passes its end goes on in the next one at a multiple of chunk, so at the same
// alignment.  flush returns whether to go on.
template <typename Size, typename Add, typename Flush>
bool adamw_pieces(int count, int64_t chunk, int max_pieces, int64_t most, Size size, Add add, Flush flush) {
    int pieces = 0;
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
        const int64_t n = size(i);
        for (int64_t at = 0; at < n;) {
            if (pieces == max_pieces || blocks == most) {
                if (!flush()) return false;
                pieces = 0;
                blocks = 0;
            }
            const int64_t left = n - at, nb = (left + chunk - 1) / chunk, take = nb <= most - blocks ? nb : most - blocks;
            const int64_t m = take == nb ? left : take * chunk;
            add(i, at, m, blocks);
            ++pieces;
            blocks += take;
            at += m;
        }
    }
    return pieces == 0 || flush();
}

}  // namespace nm
