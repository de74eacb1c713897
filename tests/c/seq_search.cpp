// The scan's search for blocks (csrc/seq_search.h) on the host: a warp's rounds with the 32 lanes in a loop, over a whole
// table of slots.
#include <algorithm>

#include "seq_search.h"

using namespace la::mixer;

namespace {
constexpr int B = 128;

SeqBlock find(const int64_t* cu, int32_t N, int64_t T, int64_t slot, int64_t beside, bool* same) {
    SlotSearch f = {0, N, true};
    while (f.n > 1) {
        uint32_t here = 0, there = 0;
        for (int lane = 0; lane < 32; ++lane) {
            if (lane * f.step() >= f.n) continue;
            const int32_t i = f.lo + lane * f.step();
            const int64_t v = cu[i] / B + i;
            here |= static_cast<uint32_t>(v <= slot) << lane;
            there |= static_cast<uint32_t>(v <= beside) << lane;
        }
        f.narrow(here, there);
    }
    *same = f.same;
    return block_of<B>(f.lo, cu[f.lo], cu[f.lo + 1], T, slot);
}
}  // namespace

// rows[slot] = sequence (-1: none), block, tokens, first token, order, last
extern "C" void seq_search_table(const int64_t* cu, int32_t N, int64_t T, int backward, int64_t (*rows)[6]) {
    for (int64_t slot = 0; slot < T / B + N; ++slot) {
        bool same;
        const SeqBlock b = find(cu, N, T, slot, slot + (backward ? 1 : -1), &same);
        const ChainPlace p = backward ? chain_place<B, true>(b.c, b.len, same) : chain_place<B, false>(b.c, b.len, same);
        const int64_t row[6] = {b.seq, b.c, b.count, b.start, p.order, p.last};
        std::copy(row, row + 6, rows[slot]);
    }
}
