// seq_search.h -- which block of which sequence a slot holds, and where the block stands in its sequence's chain: the
// arithmetic alone, one lane's or one warp's at a time, so that the host can run it too (mixer.cuh has the warp's form).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define LA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define LA_HOST_DEVICE inline
#endif

namespace la {
namespace mixer {

// The packed batch is cut into blocks of `B` tokens that start at each sequence's own first
// token, so that what a block computes does not depend on the batch around its sequence.  Block
// c of sequence i is slot cu[i] / B + i + c: these numbers are all different (a sequence of L
// tokens from cu[i] on needs at most floor((cu[i] + L) / B) - floor(cu[i] / B) + 1 of them), there
// are T / B + N slots, each sequence has at least one (an empty one too), and no table is needed.
struct SeqBlock {
    int32_t seq;    // -1: the slot holds no block
    int32_t start;  // first token of the block
    int32_t count;  // tokens in the block (0 only for the block of an empty sequence)
    int32_t c;      // block number within the sequence
    int32_t len;    // tokens in the sequence
    int32_t first;  // first token of the sequence
};

// The search for the last sequence whose first block is at or before a slot, 32 candidates a round: sequences
// [lo, lo + n) are left.  A slot `beside` it goes through the same rounds, as long as it would find the same sequence.
struct SlotSearch {
    int32_t lo, n;
    bool same;
    LA_HOST_DEVICE int32_t step() const { return (n + 31) / 32; }
    // Takes the round's answers, one bit a candidate: whether sequence lo + lane * step() begins at or before the slot,
    // and before the one beside it.
    LA_HOST_DEVICE void narrow(uint32_t here, uint32_t beside) {
        const int32_t s = step(), k = highest(here);
        same = same && k == highest(beside);
        lo += k * s;
        n = s < n - k * s ? s : n - k * s;
    }
    LA_HOST_DEVICE static int32_t highest(uint32_t m) {
#ifdef __CUDA_ARCH__
        return m ? 31 - __clz(static_cast<int>(m)) : 0;
#else
        return m ? 31 - __builtin_clz(m) : 0;
#endif
    }
};

// The block in `slot`, sequence `seq` being tokens [s0, s1).  With invalid boundaries it is none, or some block inside
// [0, T), so that no access leaves the operands.
template <int B>
LA_HOST_DEVICE SeqBlock block_of(int32_t seq, int64_t s0, int64_t s1, int64_t T, int64_t slot) {
    SeqBlock b;
    b.seq = -1;
    b.start = b.c = b.len = b.first = 0;
    b.count = 0;
    if (s0 < 0 || s1 < s0 || s1 > T) return b;
    const int64_t c = slot - (s0 / B + seq);
    if (c < 0 || (c > 0 && c * B >= s1 - s0)) return b;
    b.seq = seq;
    b.c = static_cast<int32_t>(c);
    b.first = static_cast<int32_t>(s0);
    b.len = static_cast<int32_t>(s1 - s0);
    b.start = static_cast<int32_t>(s0 + c * B);
    const int32_t rest = b.first + b.len - b.start;
    b.count = rest < B ? rest : B;
    return b;
}

// A block's place in the chain of its sequence, from the first block on or (backward) from the last.  It takes over from
// the slot beside it, before or after; where the search does not find that block there, which only invalid boundaries
// do, nobody leaves it anything and it begins a chain of its own: a block never waits for one that is not there.
struct ChainPlace {
    int32_t order;  // 0: begins the chain
    bool last;      // nobody takes over from it
};
template <int B, bool kBackward>
LA_HOST_DEVICE ChainPlace chain_place(int32_t c, int32_t len, bool chained) {
    const int32_t blocks = len > B ? (len - 1) / B + 1 : 1;
    ChainPlace p;
    p.last = c == (kBackward ? 0 : blocks - 1);
    p.order = !chained ? 0 : kBackward ? blocks - 1 - c : c;
    return p;
}

}  // namespace mixer
}  // namespace la
