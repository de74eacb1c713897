// glr.cuh -- the gated linear recurrence: what glr_fwd.cu, glr_bwd.cu and glr.cu share.
//
// Per sequence and channel, with l_t the log decay of g_t, a_t = e^{l_t} and m_t = 1 or 1 - a_t:
//
//   h_t = a_t h_{t-1} + m_t x_t
//
// and backwards, e_t being the gradient of h_t:
//
//   e_t = dh_t + a_{t+1} e_{t+1},  dx_t = m_t e_t,  dl_t = e_t a_t (h_{t-1} - [m = 1 - a] x_t),
//   dg_t = dl_t dl/dg,  d(initial) = a_1 e_1.
//
// Every step is the affine map h -> a h + u, and maps compose, so the time axis is split.  A CTA takes
// a block of 128 tokens x 64 channels into shared memory, each warp its own 16 or 32 tokens by TMA,
// each thread half of them of 4 channels.  First pass: the block's composed map.  Then one number per channel
// from the block before, the state entering it.  Second pass: the block again from shared memory (the
// gate is cheaper to evaluate twice than to keep), results over the inputs, stored by TMA.
//
// The entering states run through a table in the workspace.  A block publishes its composed map (A, B)
// as soon as it has it and the state leaving it once it knows the one entering; a block that needs a
// state looks back over up to 32 predecessors, takes the nearest published state and folds the maps
// after it in order.  The state leaving a block is always fma(A, entering, B), whoever computes it, so
// the bits do not depend on what was published when.  The launch is cooperative (all CTAs resident),
// every CTA walks its items in ascending order and items only wait for lower ones, so the lowest
// unfinished item never waits and the waits end; they are bounded all the same (LA_ERR_TIMEOUT).  Each
// operand is read once and each result written once.
//
// The backward runs the same chain from each sequence's end, over the gradient leaving a token,
// c_t = a_t (dh_t + c_{t+1}); the states entering its blocks come from the forward's checkpoints (one
// row per 128 tokens, 1.5 % of the operands' bytes), so it is one pass too.
#pragma once
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "mixer.cuh"

namespace la {
namespace glr {

using namespace la::mixer;

constexpr int kBlock = 128;                      // tokens of a block, and between saved states
constexpr int kChannels = 64;                    // of a CTA, four a lane
constexpr uint64_t kWaitNs = 1000000000ull;      // a bounded wait gives up after a second

// A CTA's kWarps warps take 128 / kWarps tokens each, half a warp half of those.
template <int kWarps>
constexpr int span() { return kBlock / kWarps / 2; }

// e^l and, for the complement, 1 - e^l, of two values.  An error in a decay near 1 adds up over some 1 / |l| tokens, by
// its mean where decays vary and whole where they stay the same.  ex2.approx is 0.3 units of 2^-24 low on average just
// below 1 (65536 logits), which its argument makes up for: means are then within 0.2 units, single values within 1.7 for
// |l| below 1/8, as good as a 32-bit exp's.  kNear: l itself is the input, and below 1/16 the Taylor series to l^4 (off by
// 8e-9) takes ex2's place, which leaves the rounding alone (0.5 units).  The bounded gate goes without: its l has
// roundings of its own, and the series takes 7 % of its dense forward's time and 12 % of its backward's.  With the
// complement the series goes to l^7 and 1/2 (2e-7 of 1 - e^l there), as the difference would cancel.
constexpr float kEx2Low = 0.3f * 0x1p-24f * kLog2e;
template <bool kComplement, bool kNear>
__device__ __forceinline__ void exp_both(float2 l, float2& e, float2& rest) {
    const float2 t = fma2(l, both(kLog2e), both(kEx2Low));
    e = make_float2(ex2(t.x), ex2(t.y));
    rest = both(1.f);
    if (!kComplement && !kNear) return;
    float2 q = both(1.f / 24.f);  // (e^l - 1) / l
    if (kComplement) {
        q = fma2(l, both(1.f / 5040.f), both(1.f / 720.f));
        q = fma2(l, q, both(1.f / 120.f));
        q = fma2(l, q, both(1.f / 24.f));
    }
    q = fma2(l, q, both(1.f / 6.f));
    q = fma2(l, q, both(0.5f));
    q = fma2(l, q, both(1.f));
    const float2 p = fma2(l, q, both(1.f));
    constexpr float kSmall = kComplement ? 0.5f : 0.0625f;
    const bool s0 = fabsf(l.x) < kSmall, s1 = fabsf(l.y) < kSmall;
    if (kComplement) {
        const float2 r = mul2(mul2(l, both(-1.f)), q), d = fma2(e, both(-1.f), both(1.f));
        rest = make_float2(s0 ? r.x : d.x, s1 ? r.y : d.y);
    }
    e = make_float2(s0 ? p.x : e.x, s1 ? p.y : e.y);
}

// a, m and dl/dg of two gate values.  s(g) = 1 / (1 + e) and 1 - s(g) = e s(g) with e = exp(-g): no cancellation.  From
// e = 2^64 on 1 - s(g) is 1 in 32 bits, and s(g) goes on to 0 while e goes on to infinity (NaN stays NaN).
struct Gated {
    float2 a, m, slope;
};
template <int kMode, bool kComplement>
__device__ __forceinline__ Gated gate(float lb, float2 g) {
    Gated r;
    float2 l = g;
    r.slope = both(1.f);
    if (kMode != LA_GATE_LOG) {
        const float2 t = mul2(g, both(-kLog2e)), e = make_float2(ex2(t.x), ex2(t.y));
        const float2 q = add2(e, both(1.f)), s = make_float2(rcp_fast(q.x), rcp_fast(q.y)), es = mul2(e, s);
        const float2 rest = make_float2(t.x > 64.f ? 1.f : es.x, t.y > 64.f ? 1.f : es.y);
        if (kMode == LA_GATE_LOGSIGMOID) {
            r.a = s;
            r.slope = rest;
            r.m = kComplement ? rest : both(1.f);
            return r;
        }
        l = mul2(both(lb), s);
        r.slope = mul2(l, rest);
    }
    exp_both<kComplement, kMode == LA_GATE_LOG>(l, r.a, r.m);
    return r;
}

// Calls f with the gate's mode and complement as constants.
template <int kMode, bool kComplement>
struct Gate {
    static constexpr int mode = kMode;
    static constexpr bool complement = kComplement;
};
template <typename F>
__host__ __device__ __forceinline__ void with_gate(int mode, int complement, F f) {
    if (mode == LA_GATE_LOG) complement ? f(Gate<LA_GATE_LOG, true>()) : f(Gate<LA_GATE_LOG, false>());
    else if (mode == LA_GATE_LOGSIGMOID) complement ? f(Gate<LA_GATE_LOGSIGMOID, true>()) : f(Gate<LA_GATE_LOGSIGMOID, false>());
    else complement ? f(Gate<LA_GATE_SIGMOID_BOUND, true>()) : f(Gate<LA_GATE_SIGMOID_BOUND, false>());
}

struct Args {
    const void *x, *g, *cu, *s0;
    int64_t x_st, g_st, T;
    int cu64, N, D, mode, compl_in, s0_bf16;
    float lb;
    const int32_t* idx;
    int64_t pool;
    void* h;
    int64_t h_st;
    float *fin, *ckpt;
    const void* dh;
    const float* dfin;
    void *dx, *dg;
    int64_t dh_st, dx_st, dg_st;
    float* ds0;
    int32_t* status;
    int tiles;         // channel tiles
    int64_t items;     // (T / kBlock + N) * tiles
    ulonglong2* maps;  // [slots][tiles][32]: (A, B) of a lane's two channels; null when no sequence has two blocks
    uint2* states;     // [slots][tiles][32]: the states leaving the block
    int tma;           // every operand can move by TMA
};

// Calls f with a constant that says whether the thread's span is whole, as all but a sequence's last are: its loops
// then have no bounds to check.
template <int kSpan, typename F>
__device__ __forceinline__ void with_span(int n, F f) {
    if (n >= kSpan) f(std::true_type());
    else f(std::false_type());
}

// ---------------------------------------------------------------- a thread's four channels of one row in shared memory
struct Four {
    float2 v[2];
};
template <typename T>
__device__ __forceinline__ Four get4(const T* p) {
    Four r;
    if (sizeof(T) == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        r.v[0] = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
        r.v[1] = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        const float4 w = *reinterpret_cast<const float4*>(p);
        r.v[0] = make_float2(w.x, w.y);
        r.v[1] = make_float2(w.z, w.w);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void put4(T* p, const Four& f) {
    if (sizeof(T) == 2) {
        __nv_bfloat162 lo = __floats2bfloat162_rn(f.v[0].x, f.v[0].y), hi = __floats2bfloat162_rn(f.v[1].x, f.v[1].y);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
    }
}
__device__ __forceinline__ Four four(float x) { return {{both(x), both(x)}}; }
__device__ __forceinline__ Four fma4(const Four& a, const Four& b, const Four& c) {
    return {{fma2(a.v[0], b.v[0], c.v[0]), fma2(a.v[1], b.v[1], c.v[1])}};
}
__device__ __forceinline__ Four mul4(const Four& a, const Four& b) { return {{mul2(a.v[0], b.v[0]), mul2(a.v[1], b.v[1])}}; }
__device__ __forceinline__ Four other_half(const Four& a) {
    return {{make_float2(__shfl_xor_sync(0xffffffffu, a.v[0].x, 16), __shfl_xor_sync(0xffffffffu, a.v[0].y, 16)),
             make_float2(__shfl_xor_sync(0xffffffffu, a.v[1].x, 16), __shfl_xor_sync(0xffffffffu, a.v[1].y, 16))}};
}

// ---------------------------------------------------------------- a warp's rows between global and shared memory
// Without TMA: lane by lane, rows [0, n) of the warp, channels below D.
template <typename T>
__device__ __forceinline__ void rows_in(T* s, const void* base, int64_t stride, int64_t token, int n, int d, int D) {
    const int lane = threadIdx.x & 31;
    const T* p = static_cast<const T*>(base) + token * stride + d;
#pragma unroll 8
    for (int r = 0; r < n; ++r)
#pragma unroll
        for (int c = 0; c < kChannels; c += 32) s[r * kChannels + c + lane] = d + c + lane < D ? p[r * stride + c + lane] : from_f<T>(0.f);
}
template <typename T>
__device__ __forceinline__ void rows_out(const T* s, void* base, int64_t stride, int64_t token, int n, int d, int D) {
    const int lane = threadIdx.x & 31;
    T* p = static_cast<T*>(base) + token * stride + d;
    for (int r = 0; r < n; ++r)
#pragma unroll
        for (int c = 0; c < kChannels; c += 32)
            if (d + c + lane < D) p[r * stride + c + lane] = s[r * kChannels + c + lane];
}

__device__ __forceinline__ void load2_any(const void* base, int64_t at, int d, int D, int is_bf16, float& v0, float& v1) {
    v0 = d < D ? load_any(base, at + d, is_bf16) : 0.f;
    v1 = d + 1 < D ? load_any(base, at + d + 1, is_bf16) : 0.f;
}
__device__ __forceinline__ void store2_any(void* base, int64_t at, int d, int D, int is_bf16, float v0, float v1) {
    if (d < D) store_any(base, at + d, is_bf16, v0);
    if (d + 1 < D) store_any(base, at + d + 1, is_bf16, v1);
}

// ---------------------------------------------------------------- items and the chain between them
// Item j is channel tile j mod tiles of a block.  Up to 32 sequences are taken side by side, first the first block
// of each (the last, in the backward), then the second of each that has one, and so on: the state that a block needs
// was then published a round of items earlier, and is read ahead of its rows (`peek`).  More sequences, and a single
// one, go slot by slot.  Either way a block comes after the one whose state it needs, its neighbour in the table of
// slots.
struct Item {
    int32_t start, count;  // tokens of the block
    int32_t d;             // first channel
    int32_t order;         // place in the sequence's chain: 0 needs no neighbour
    int32_t slot;          // block slot (the checkpoint row); its words in the table: slot * tiles + tile
    int32_t state;         // row of the initial state
    int32_t tile;
    bool last, dead;       // end of the chain; nothing to do (no block, or a bad state index)
};

// By a whole warp.
template <bool kBackward>
__device__ __forceinline__ void locate(const Args& a, int64_t j, Item* to) {
    const int lane = threadIdx.x & 31;
    Item it;
    const int32_t s = static_cast<int32_t>(j / a.tiles);
    it.tile = static_cast<int32_t>(j - static_cast<int64_t>(s) * a.tiles);
    it.d = it.tile * kChannels;
    it.slot = it.count = 0;
    int32_t seq = -1, start = 0, len = 0, c = 0;
    bool chained = true;  // the neighbour holds the block that this one follows (invalid boundaries may leave it none)
    if (a.N > 1 && a.N <= 32) {
        // lane i holds sequence i; the blocks of rounds before round r are sum_i min(blocks_i, r)
        int64_t s0 = 0, s1 = -1;
        if (lane < a.N) {
            s0 = cu_load(a.cu, a.cu64, lane);
            s1 = cu_load(a.cu, a.cu64, lane + 1);
        }
        const bool valid = s0 >= 0 && s1 >= s0 && s1 <= a.T;
        const uint32_t mine = valid ? max(1u, static_cast<uint32_t>((s1 - s0 + kBlock - 1) / kBlock)) : 0u;
        uint32_t lo = 0, hi = __reduce_max_sync(0xffffffffu, mine), before = 0;
        while (lo < hi) {  // the last round that begins at or before block s
            const uint32_t mid = (lo + hi + 1) / 2, sum = __reduce_add_sync(0xffffffffu, min(mine, mid));
            if (sum <= static_cast<uint32_t>(s)) {
                lo = mid;
                before = sum;
            } else {
                hi = mid - 1;
            }
        }
        const unsigned in_round = __ballot_sync(0xffffffffu, mine > lo);
        const int nth = static_cast<int>(s - before) + 1;  // of those that have this round
        const bool chosen = (in_round >> lane & 1u) && __popc(in_round & ((2u << lane) - 1u)) == nth;
        const unsigned who = __ballot_sync(0xffffffffu, chosen);
        if (who) {
            seq = __ffs(who) - 1;
            const int32_t first = __shfl_sync(0xffffffffu, static_cast<int32_t>(s0), seq);
            len = __shfl_sync(0xffffffffu, static_cast<int32_t>(s1 - s0), seq);
            const int32_t blocks = static_cast<int32_t>(__shfl_sync(0xffffffffu, mine, seq));
            c = kBackward ? blocks - 1 - static_cast<int32_t>(lo) : static_cast<int32_t>(lo);
            start = first + c * kBlock;
            it.slot = first / kBlock + seq + c;
            it.count = min(kBlock, first + len - start);
        }
    } else {
        it.slot = kBackward ? static_cast<int32_t>(a.T / kBlock) + a.N - 1 - s : s;
        const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, it.slot, it.slot + (kBackward ? 1 : -1), chained);
        seq = b.seq;
        start = b.start;
        len = b.len;
        c = b.c;
        it.count = b.count;
    }
    it.start = start;
    it.dead = seq < 0;
    const ChainPlace place = chain_place<kBlock, kBackward>(c, len, chained);
    it.order = place.order;
    it.last = place.last;
    it.state = seq;
    if (!kBackward && a.idx && !it.dead) {
        it.state = a.idx[seq];
        if (it.state < 0 || it.state >= a.pool) {
            raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
            it.dead = true;
        }
    }
    if (it.dead) it.count = 0;
    if (lane == 0) *to = it;
    __syncwarp();
}

// The chain's words carry their own readiness, so that neither side needs a fence: a map (A, B) is one
// 64-bit word and a state one 32-bit word, each written by a single store (16-byte and 8-byte vectors
// hold a lane's two channels, every element of its own).  The table starts as all ones, a NaN that
// `settled` keeps out of what is published.
constexpr uint32_t kUnset = 0xFFFFFFFFu;
__device__ __forceinline__ float settled(float x) { return __float_as_uint(x) == kUnset ? __uint_as_float(0x7FC00000u) : x; }

__device__ __forceinline__ uint2 load_state(const uint2* p) {
    uint2 v;
    asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ ulonglong2 load_map(const ulonglong2* p) {
    ulonglong2 v;
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void publish_state(uint2* p, float2 v) {
    asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(__float_as_uint(settled(v.x))),
                 "r"(__float_as_uint(settled(v.y)))
                 : "memory");
}
__device__ __forceinline__ unsigned long long word(float a, float b) {
    return static_cast<unsigned long long>(__float_as_uint(settled(a))) |
           (static_cast<unsigned long long>(__float_as_uint(b)) << 32);
}
__device__ __forceinline__ void publish_map(ulonglong2* p, float4 m) {
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(word(m.x, m.z)), "l"(word(m.y, m.w)) : "memory");
}

// The state entering the block with words w for this lane's two channels: the nearest published state among up to
// kWindow predecessors that only published maps lie after, with those maps folded in order.  The
// window's words are read together.  A wait over a second gives up (status).
constexpr int kWindow = 32, kBatch = 4;
template <bool kBackward>
__device__ __forceinline__ float2 look_back(const Args& a, int64_t w, int32_t order) {
    const int lane = threadIdx.x & 31;
    const int n = min(order, kWindow);
    const int64_t stride = (kBackward ? -32 : 32) * static_cast<int64_t>(a.tiles);
    const uint2* states = a.states + w * 32 + lane - stride;  // the predecessor's, and back from it
    const ulonglong2* maps = a.maps + w * 32 + lane - stride;
    uint64_t t0 = 0;
    float2 h = make_float2(0.f, 0.f);
    int k = 0, found = -1;  // the nearest k predecessors have published maps, but no state when last looked at
    for (int spin = 0; found < 0; ++spin) {
        uint2 s[kBatch];
        ulonglong2 m[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int q = min(k + i, n - 1);
            s[i] = load_state(states - q * stride);
            m[i] = load_map(maps - q * stride);
        }
        bool open = true;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (!open || k >= n) continue;
            if (s[i].x != kUnset && s[i].y != kUnset) {
                h = make_float2(__uint_as_float(s[i].x), __uint_as_float(s[i].y));
                found = k;
                open = false;
            } else if (static_cast<uint32_t>(m[i].x) != kUnset && static_cast<uint32_t>(m[i].y) != kUnset && k + 1 < n) {
                ++k;
            } else {
                open = false;
                k = 0;  // look again from the nearest
            }
        }
        if (found < 0 && (spin & 255) == 255) {
            uint64_t now;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
            if (!t0) t0 = now;
            if (now - t0 > kWaitNs) {
                raise_status(a.status, LA_ERR_TIMEOUT);
                return h;
            }
        }
    }
    for (int i = found - 1; i >= 0; i -= kBatch) {
        ulonglong2 m[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) m[q] = load_map(maps - max(i - q, 0) * stride);
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            if (i - q >= 0) {
                h.x = fmaf(__uint_as_float(static_cast<uint32_t>(m[q].x)), h.x, __uint_as_float(static_cast<uint32_t>(m[q].x >> 32)));
                h.y = fmaf(__uint_as_float(static_cast<uint32_t>(m[q].y)), h.y, __uint_as_float(static_cast<uint32_t>(m[q].y >> 32)));
            }
    }
    return h;
}

__device__ __forceinline__ int64_t words_of(const Args& a, const Item& it) {
    return static_cast<int64_t>(it.slot) * a.tiles + it.tile;
}
// The predecessor's state if it is there already (unset words otherwise, and where there is none).
template <bool kBackward>
__device__ __forceinline__ uint2 peek(const Args& a, const Item& it) {
    if (it.dead || it.order == 0) return make_uint2(kUnset, kUnset);
    return load_state(a.states + (words_of(a, it) + (kBackward ? a.tiles : -a.tiles)) * 32 + (threadIdx.x & 31));
}

// One warp: finds the entering state (`in` where the chain begins; what `peek` saw; or by looking back, for which the
// item's map is published first) and publishes the leaving one.  Nobody waits for a dead item.
template <bool kBackward>
__device__ __forceinline__ void chain(const Args& a, const Item& it, float4 map, uint2 seen, float2& in, float2& out) {
    const int lane = threadIdx.x & 31;
    if (it.dead) return;
    const int64_t w = words_of(a, it);
    map.x = settled(map.x);
    map.y = settled(map.y);
    if (it.order > 0) {
        if (__all_sync(0xffffffffu, seen.x != kUnset && seen.y != kUnset)) {
            in = make_float2(__uint_as_float(seen.x), __uint_as_float(seen.y));
        } else {
            if (!it.last) publish_map(a.maps + w * 32 + lane, map);
            in = look_back<kBackward>(a, w, it.order);
        }
    }
    out = make_float2(fmaf(map.x, in.x, map.z), fmaf(map.y, in.y, map.w));
    if (a.states && !it.last) publish_state(a.states + w * 32 + lane, out);
}

__device__ __forceinline__ void check_boundaries(const Args& a) {
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < a.N;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
}

struct Maps {
    CUtensorMap x, g, dh, out, dg;  // out: h, or dx in the backward
};

// What a scan keeps beside the staged rows.
template <int kWarps, bool kBackward>
struct Shared {
    alignas(16) float a[kWarps][kChannels], u[kWarps][kChannels];  // each warp's map
    alignas(16) float c[kBackward ? kWarps : 1][kChannels];        // and the gradients'
    alignas(16) float in[kChannels], h0[kBackward ? kChannels : 4];
    uint64_t bar[kWarps];
    Item items[2];
};

template <typename X, typename G, int kX>
constexpr size_t stage_bytes() { return static_cast<size_t>(kBlock) * kChannels * (kX * sizeof(X) + sizeof(G)); }

// CTAs that an SM of the current device holds of a kernel (0: an error), looked up once per device.
template <auto kKernel>
int resident_ctas(int dev, int threads, size_t smem) {
    static std::atomic<int> known[128];
    if (dev < 0 || dev >= 128) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kKernel, threads, smem) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            return 0;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <auto kKernel>
la_status launch_scan(int threads, size_t smem, Args& a, Maps& maps, cudaStream_t s) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return LA_ERR_CUDA;
    const int per_sm = resident_ctas<kKernel>(dev, threads, smem);
    if (per_sm == 0) return LA_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.items, static_cast<int64_t>(sms) * per_sm));
    void* args[] = {&a, &maps};
    if (cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kKernel), dim3(grid), dim3(threads), args, smem, s) != cudaSuccess) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    return LA_OK;
}

// The scans, for every type and gate; the caller has set up a but for its tma.
la_status run_fwd(Args& a, int32_t x_dtype, int32_t g_dtype, cudaStream_t s);
la_status run_bwd(Args& a, int32_t x_dtype, int32_t g_dtype, cudaStream_t s);

// A map of one operand's tiles (one warp's rows); false where TMA cannot move them.
inline bool row_map(CUtensorMap* m, const Args& a, const void* p, int64_t stride, int32_t dtype, int rows) {
    return tileable(p, stride, a.T, a.D, dtype) && tile_map(m, p, stride, a.T, a.D, dtype, kChannels, rows);
}

}  // namespace glr
}  // namespace la
