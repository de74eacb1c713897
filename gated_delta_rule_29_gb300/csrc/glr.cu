// glr.cu -- the gated linear recurrence (glr_fwd, glr_bwd, glr_decode).
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
// a block of 128 tokens x 64 channels into shared memory, each warp its own 16 tokens by TMA, each
// thread 8 tokens of 4 channels.  First pass: the block's composed map.  Then one number per channel
// from the block before, the state entering it.  Second pass: the block again from shared memory (the
// gate is cheaper to evaluate twice than to keep), results over the inputs, stored by TMA.
//
// The entering states run through a table in the workspace.  A block publishes its composed map (A, B)
// as soon as it has it and the state leaving it once it knows the one entering; a block that needs a
// state looks back over up to 32 predecessors, takes the nearest published state and folds the maps
// after it in order.  The state leaving a block is always fma(A, entering, B), whoever computes it, so
// the bits do not depend on what was published when.  The launch is cooperative (all CTAs resident),
// every CTA walks its items in ascending order and items only wait for lower ones, so the lowest
// unfinished item never waits and the waits end; they are bounded all the same.  Each operand is read
// once and each result written once.
//
// The backward runs the same chain from each sequence's end, over the gradient leaving a token,
// c_t = a_t (dh_t + c_{t+1}); the states entering its blocks come from the forward's checkpoints (one
// row per 128 tokens, 1.5 % of the operands' bytes), so it is one pass too.
#include <algorithm>

#include "mixer.cuh"

namespace {

using namespace la;
using namespace la::mixer;

constexpr int kThreads = 128;                    // decode
constexpr int kWarps = 8;                        // of a scan CTA
constexpr int kScanThreads = 32 * kWarps;
constexpr int kSpan = 8;                         // tokens of a thread
constexpr int kWarpRows = 2 * kSpan;             // tokens of a warp: its halves take one span each
constexpr int kBlock = kWarpRows * kWarps;       // tokens of a block, and between saved states
constexpr int kChannels = 64;                    // of a CTA, four a lane
constexpr uint64_t kWaitNs = 1000000000ull;      // a bounded wait gives up after a second
static_assert(kBlock == 128, "the checkpoint cadence of the interface");

// e^l as 2^(l log2 e): the product's rounding is off by |l| 2^-24 of the result, which is small where
// the result is not; results below 2^-126 are zero.
__device__ __forceinline__ float exp_fast(float l) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(l * 1.4426950408889634f));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 - e^l given e^l: the Taylor series (to l^7 / 7!, 2e-7 of it at 1/2) where the difference would cancel.
__device__ __forceinline__ float one_minus_exp(float l, float e) {
    float p = fmaf(l, 1.f / 7.f, 1.f);
    p = fmaf(l * (1.f / 6.f), p, 1.f);
    p = fmaf(l * (1.f / 5.f), p, 1.f);
    p = fmaf(l * (1.f / 4.f), p, 1.f);
    p = fmaf(l * (1.f / 3.f), p, 1.f);
    p = fmaf(l * (1.f / 2.f), p, 1.f);
    return fabsf(l) < 0.5f ? -l * p : 1.f - e;
}

// a, m and dl/dg of one gate value.  s(g) and 1 - s(g) come from e = exp(-|g|) without cancellation.
template <int kMode, bool kComplement>
__device__ __forceinline__ void gate(float lb, float g, float& a, float& m, float& slope) {
    float l = g;
    slope = 1.f;
    if (kMode != LA_GATE_LOG) {
        const float e = exp_fast(-fabsf(g)), big = rcp_fast(1.f + e), small = e * big;
        const float s = g >= 0.f ? big : small, rest = g >= 0.f ? small : big;
        if (kMode == LA_GATE_LOGSIGMOID) {
            a = s;
            slope = rest;
            m = kComplement ? rest : 1.f;
            return;
        }
        l = lb * s;
        slope = l * rest;
    }
    a = exp_fast(l);
    m = kComplement ? one_minus_exp(l, a) : 1.f;
}

// Calls f with the gate's mode and complement as constants.
template <int kMode, bool kComplement>
struct Gate {
    static constexpr int mode = kMode;
    static constexpr bool complement = kComplement;
};
template <typename F>
__device__ __forceinline__ void with_gate(int mode, int complement, F f) {
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
    ulonglong2* maps;  // [items][32]: (A, B) of a lane's two channels; null when no sequence has two blocks
    uint2* states;     // [items][32]: the states leaving the item
    int tma;           // every operand can move by TMA
};

// ---------------------------------------------------------------- a thread's four channels of one row in shared memory
template <typename T>
__device__ __forceinline__ void get4(const T* p, float (&v)[4]) {
    if (sizeof(T) == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        v[0] = __uint_as_float(w.x << 16);
        v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(w.y << 16);
        v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
        const float4 w = *reinterpret_cast<const float4*>(p);
        v[0] = w.x;
        v[1] = w.y;
        v[2] = w.z;
        v[3] = w.w;
    }
}
template <typename T>
__device__ __forceinline__ void put4(T* p, const float (&v)[4]) {
    if (sizeof(T) == 2) {
        __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
}
// Two of the four channels (p points at the first of the pair).
template <typename T>
__device__ __forceinline__ float2 get2(const T* p) {
    if (sizeof(T) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    return *reinterpret_cast<const float2*>(p);
}
template <typename T>
__device__ __forceinline__ void put2(T* p, float x, float y) {
    if (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
    else *reinterpret_cast<float2*>(p) = make_float2(x, y);
}

// ---------------------------------------------------------------- a warp's rows between global and shared memory
// Without TMA: lane by lane, rows [0, n) of the warp, channels below D.
template <typename T>
__device__ __forceinline__ void rows_in(T* s, const void* base, int64_t stride, int64_t token, int n, int d, int D) {
    const int lane = threadIdx.x & 31;
    const T* p = static_cast<const T*>(base) + token * stride + d;
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
// Item j is block `slot` and channel tile j mod tiles; slots ascend in the forward and descend in the
// backward, so that the neighbour whose state an item needs is item j - tiles.
struct Item {
    int32_t start, count;  // tokens of the block
    int32_t d;             // first channel
    int32_t order;         // place in the sequence's chain: 0 needs no neighbour
    int32_t slot;          // block slot (the checkpoint row)
    int32_t state;         // row of the initial state
    bool last, dead;       // end of the chain; nothing to do (no block, or a bad state index)
};

// By a whole warp.
template <bool kBackward>
__device__ __forceinline__ void locate(const Args& a, int64_t j, Item* to) {
    Item it;
    const int32_t s = static_cast<int32_t>(j / a.tiles);
    it.slot = kBackward ? static_cast<int32_t>(a.T / kBlock) + a.N - 1 - s : s;
    it.d = static_cast<int32_t>(j - static_cast<int64_t>(s) * a.tiles) * kChannels;
    const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, it.slot);
    it.start = b.start;
    it.count = b.count;
    it.dead = b.seq < 0;
    const int32_t blocks = max(1, (b.len + kBlock - 1) / kBlock);
    it.order = kBackward ? blocks - 1 - b.c : b.c;
    it.last = it.order == blocks - 1;
    it.state = b.seq;
    if (!kBackward && a.idx && !it.dead) {
        it.state = a.idx[b.seq];
        if (it.state < 0 || it.state >= a.pool) {
            raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
            it.dead = true;
        }
    }
    if (it.dead) it.count = 0;
    if ((threadIdx.x & 31) == 0) *to = it;
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

// The state entering item j for this lane's two channels: the nearest published state among up to
// kWindow predecessors that only published maps lie after, with those maps folded in order.  The
// window's words are read together.  A wait over a second gives up (status).
constexpr int kWindow = 32, kBatch = 4;
__device__ __forceinline__ float2 look_back(const Args& a, int64_t j, int32_t order) {
    const int lane = threadIdx.x & 31;
    const int n = min(order, kWindow);
    const int64_t stride = static_cast<int64_t>(a.tiles) * 32;
    const uint2* states = a.states + (j - a.tiles) * 32 + lane;      // the predecessor's, and back from it
    const ulonglong2* maps = a.maps + (j - a.tiles) * 32 + lane;
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

// One warp: publishes the item's map, finds the entering state (`in` where the chain begins), publishes
// the leaving one.
__device__ __forceinline__ void chain(const Args& a, int64_t j, const Item& it, float4 map, float2& in, float2& out) {
    const int lane = threadIdx.x & 31;
    if (it.dead) {
        if (a.states) publish_state(a.states + j * 32 + lane, make_float2(0.f, 0.f));
        return;
    }
    map.x = settled(map.x);
    map.y = settled(map.y);
    if (it.order > 0) {
        if (!it.last) publish_map(a.maps + j * 32 + lane, map);
        in = look_back(a, j, it.order);
    }
    out = make_float2(fmaf(map.x, in.x, map.z), fmaf(map.y, in.y, map.w));
    if (a.states && !it.last) publish_state(a.states + j * 32 + lane, out);
}

__device__ __forceinline__ void check_boundaries(const Args& a) {
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kScanThreads) + threadIdx.x; i < a.N;
         i += static_cast<int64_t>(gridDim.x) * kScanThreads)
        check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
}

struct Maps {
    CUtensorMap x, g, dh, out, dg;  // out: h, or dx in the backward
};

// What both directions keep beside the staged rows.
struct Shared {
    float a[kWarps][kChannels], u[kWarps][kChannels], c[kWarps][kChannels];  // each warp's map (c: the gradients')
    float in[kChannels], h0[kChannels];
    uint64_t bar[kWarps];
    Item items[2];
};

template <typename X, typename G, int kX>
constexpr size_t stage_bytes() { return static_cast<size_t>(kBlock) * kChannels * (kX * sizeof(X) + sizeof(G)); }

// CTAs of an SM: as many as the staged rows leave room for.
template <typename X, typename G>
constexpr int fwd_ctas() { return sizeof(X) + sizeof(G) == 4 ? 5 : sizeof(X) + sizeof(G) == 6 ? 4 : 3; }
template <typename X, typename G>
constexpr int bwd_ctas() { return sizeof(X) + sizeof(G) == 8 ? 2 : 3; }

template <typename X, typename G>
__global__ void __launch_bounds__(kScanThreads, (fwd_ctas<X, G>())) glr_fwd_kernel(const Args a, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(128) uint8_t stage[];
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = lane >> 4, c4 = (lane & 15) * 4;
    X* wx = reinterpret_cast<X*>(stage) + w * kWarpRows * kChannels;                       // the warp's rows
    G* wg = reinterpret_cast<G*>(stage + sizeof(X) * kBlock * kChannels) + w * kWarpRows * kChannels;
    X* sx = wx + half * kSpan * kChannels + c4;                                            // the thread's
    G* sg = wg + half * kSpan * kChannels + c4;
    if (lane == 0) mbar_init(&sh.bar[w], 1);
    fence_mbar_init();
    check_boundaries(a);

    // The warp's rows of an item on their way into shared memory; false when it has none.
    auto fetch = [&](const Item& it) {
        const int n = min(it.count - w * kWarpRows, kWarpRows), token = it.start + w * kWarpRows;
        if (n <= 0) return;
        if (a.tma) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&sh.bar[w], kWarpRows * kChannels * (sizeof(X) + sizeof(G)));
                tile_load(wx, &maps.x, &sh.bar[w], it.d, token);
                tile_load(wg, &maps.g, &sh.bar[w], it.d, token);
            }
        } else {
            rows_in(wx, a.x, a.x_st, token, n, it.d, a.D);
            rows_in(wg, a.g, a.g_st, token, n, it.d, a.D);
        }
    };

    int64_t j = blockIdx.x;
    uint32_t parity = 0;
    if (w == 0) locate<false>(a, j, &sh.items[0]);
    __syncthreads();
    fetch(sh.items[0]);
    for (int at = 0;; at ^= 1) {
        const Item& it = sh.items[at];
        const int64_t jn = j + gridDim.x;
        const int rows = min(it.count - w * kWarpRows, kWarpRows);  // of the warp
        const int n = rows - half * kSpan;                          // of the thread (may exceed kSpan)
        float2 in = make_float2(0.f, 0.f);
        if (w == 0 && it.order == 0 && !it.dead && a.s0)
            load2_any(a.s0, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, a.s0_bf16, in.x, in.y);
        __syncwarp();
        if (a.tma && rows > 0) {
            if (!mbar_wait(&sh.bar[w], parity, kWaitNs)) raise_status(a.status, LA_ERR_TIMEOUT);
            parity ^= 1;
        }
        // the map of the thread's span
        float ca[4] = {1.f, 1.f, 1.f, 1.f}, cu[4] = {0.f, 0.f, 0.f, 0.f};
        with_gate(a.mode, a.compl_in, [&](auto gt) {
#pragma unroll
            for (int k = 0; k < kSpan; ++k)
                if (k < n) {
                    float x[4], g[4];
                    get4(sx + k * kChannels, x);
                    get4(sg + k * kChannels, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float dec, m, slope;
                        gate<decltype(gt)::mode, decltype(gt)::complement>(a.lb, g[i], dec, m, slope);
                        cu[i] = fmaf(dec, cu[i], decltype(gt)::complement ? m * x[i] : x[i]);
                        ca[i] *= dec;
                    }
                }
        });
        // the other half's: the lower one's map enters the upper one, both make the warp's
        float oa[4], ou[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            oa[i] = __shfl_xor_sync(0xffffffffu, ca[i], 16);
            ou[i] = __shfl_xor_sync(0xffffffffu, cu[i], 16);
        }
        if (half == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sh.a[w][c4 + i] = ca[i] * oa[i];
                sh.u[w][c4 + i] = fmaf(oa[i], cu[i], ou[i]);
            }
        }
        __syncthreads();
        if (w == kWarps - 1 && jn < a.items) locate<false>(a, jn, &sh.items[at ^ 1]);
        if (w == 0) {
            float4 map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 qa = *reinterpret_cast<const float2*>(&sh.a[i][2 * lane]), qu = *reinterpret_cast<const float2*>(&sh.u[i][2 * lane]);
                map.z = fmaf(qa.x, map.z, qu.x);
                map.w = fmaf(qa.y, map.w, qu.y);
                map.x *= qa.x;
                map.y *= qa.y;
            }
            float2 out;
            chain(a, j, it, map, in, out);
            *reinterpret_cast<float2*>(&sh.in[2 * lane]) = in;
            if (!it.dead) {
                if (a.ckpt && it.count > 0) store2_any(a.ckpt, it.slot * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, in.x, in.y);
                if (it.last) {
                    if (a.idx) store2_any(const_cast<void*>(a.s0), it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, a.s0_bf16, out.x, out.y);
                    else if (a.fin) store2_any(a.fin, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, out.x, out.y);
                }
            }
        }
        // while the chain goes on: the map of the rows before this warp's (the thread's, in the upper half)
        float pa[4] = {1.f, 1.f, 1.f, 1.f}, pu[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < w; ++i) {
            float qa[4], qu[4];
            get4(&sh.a[i][c4], qa);
            get4(&sh.u[i][c4], qu);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pu[e] = fmaf(qa[e], pu[e], qu[e]);
                pa[e] *= qa[e];
            }
        }
        if (half == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pu[e] = fmaf(oa[e], pu[e], ou[e]);
                pa[e] *= oa[e];
            }
        }
        __syncthreads();
        if (a.h && rows > 0) {
            float h[4];
            get4(&sh.in[c4], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = fmaf(pa[e], h[e], pu[e]);
            with_gate(a.mode, a.compl_in, [&](auto gt) {
#pragma unroll
                for (int k = 0; k < kSpan; ++k)
                    if (k < n) {
                        float x[4], g[4];
                        get4(sx + k * kChannels, x);
                        get4(sg + k * kChannels, g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float dec, m, slope;
                            gate<decltype(gt)::mode, decltype(gt)::complement>(a.lb, g[i], dec, m, slope);
                            h[i] = fmaf(dec, h[i], decltype(gt)::complement ? m * x[i] : x[i]);
                        }
                        put4(sx + k * kChannels, h);
                    }
            });
            // whole tiles by TMA; the last rows of a sequence one by one
            if (a.tma && rows == kWarpRows) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tile_store(&maps.out, wx, it.d, it.start + w * kWarpRows);
                    bulk_commit_group();
                    bulk_wait_read_all();
                }
            } else {
                __syncwarp();
                rows_out(wx, a.h, a.h_st, it.start + w * kWarpRows, rows, it.d, a.D);
            }
        }
        if (jn >= a.items) break;
        fence_proxy_async_smem();  // the rows were written here, and are about to be by TMA
        __syncwarp();
        fetch(sh.items[at ^ 1]);
        j = jn;
    }
    if (lane == 0) bulk_wait_all();
}

template <typename X, typename G>
__global__ void __launch_bounds__(kScanThreads, (bwd_ctas<X, G>())) glr_bwd_kernel(const Args a, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(128) uint8_t stage[];
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = lane >> 4, c4 = (lane & 15) * 4;
    constexpr int kPlane = kBlock * kChannels;
    X* wx = reinterpret_cast<X*>(stage) + w * kWarpRows * kChannels;
    X* wd = wx + kPlane;
    G* wg = reinterpret_cast<G*>(stage + 2 * sizeof(X) * kPlane) + w * kWarpRows * kChannels;
    const int mine = half * kSpan * kChannels + c4;  // the thread's first element of the warp's rows
    if (lane == 0) mbar_init(&sh.bar[w], 1);
    fence_mbar_init();
    check_boundaries(a);

    auto fetch = [&](const Item& it) {
        const int n = min(it.count - w * kWarpRows, kWarpRows), token = it.start + w * kWarpRows;
        if (n <= 0) return;
        if (a.tma) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&sh.bar[w], kWarpRows * kChannels * (2 * sizeof(X) + sizeof(G)));
                tile_load(wx, &maps.x, &sh.bar[w], it.d, token);
                tile_load(wd, &maps.dh, &sh.bar[w], it.d, token);
                tile_load(wg, &maps.g, &sh.bar[w], it.d, token);
            }
        } else {
            rows_in(wx, a.x, a.x_st, token, n, it.d, a.D);
            rows_in(wd, a.dh, a.dh_st, token, n, it.d, a.D);
            rows_in(wg, a.g, a.g_st, token, n, it.d, a.D);
        }
    };

    int64_t j = blockIdx.x;
    uint32_t parity = 0;
    if (w == 0) locate<true>(a, j, &sh.items[0]);
    __syncthreads();
    fetch(sh.items[0]);
    for (int at = 0;; at ^= 1) {
        const Item& it = sh.items[at];
        const int64_t jn = j + gridDim.x;
        const int rows = min(it.count - w * kWarpRows, kWarpRows);
        const int n = rows - half * kSpan;
        float2 in = make_float2(0.f, 0.f);
        if (w == 0 && it.order == 0 && !it.dead && a.dfin)
            load2_any(a.dfin, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, in.x, in.y);
        if (w == 1 && it.count > 0) load2_any(a.ckpt, it.slot * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, in.x, in.y);
        __syncwarp();
        if (a.tma && rows > 0) {
            if (!mbar_wait(&sh.bar[w], parity, kWaitNs)) raise_status(a.status, LA_ERR_TIMEOUT);
            parity ^= 1;
        }
        // the maps of the thread's span, h -> ca h + cu forwards and c -> ca c + cc backwards
        float ca[4] = {1.f, 1.f, 1.f, 1.f}, cu[4] = {0.f, 0.f, 0.f, 0.f}, cc[4] = {0.f, 0.f, 0.f, 0.f};
        with_gate(a.mode, a.compl_in, [&](auto gt) {
#pragma unroll
            for (int k = 0; k < kSpan; ++k)
                if (k < n) {
                    float x[4], g[4], d[4];
                    get4(wx + mine + k * kChannels, x);
                    get4(wg + mine + k * kChannels, g);
                    get4(wd + mine + k * kChannels, d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float dec, m, slope;
                        gate<decltype(gt)::mode, decltype(gt)::complement>(a.lb, g[i], dec, m, slope);
                        cu[i] = fmaf(dec, cu[i], decltype(gt)::complement ? m * x[i] : x[i]);
                        ca[i] *= dec;
                        cc[i] = fmaf(ca[i], d[i], cc[i]);
                    }
                }
        });
        float oa[4], ou[4], oc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            oa[i] = __shfl_xor_sync(0xffffffffu, ca[i], 16);
            ou[i] = __shfl_xor_sync(0xffffffffu, cu[i], 16);
            oc[i] = __shfl_xor_sync(0xffffffffu, cc[i], 16);
        }
        if (half == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sh.a[w][c4 + i] = ca[i] * oa[i];
                sh.u[w][c4 + i] = fmaf(oa[i], cu[i], ou[i]);
                sh.c[w][c4 + i] = fmaf(ca[i], oc[i], cc[i]);
            }
        }
        if (w == 1) *reinterpret_cast<float2*>(&sh.h0[2 * lane]) = in;
        __syncthreads();
        if (w == kWarps - 1 && jn < a.items) locate<true>(a, jn, &sh.items[at ^ 1]);
        if (w == 0) {
            float4 map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 qa = *reinterpret_cast<const float2*>(&sh.a[i][2 * lane]), qc = *reinterpret_cast<const float2*>(&sh.c[i][2 * lane]);
                map.z = fmaf(map.x, qc.x, map.z);
                map.w = fmaf(map.y, qc.y, map.w);
                map.x *= qa.x;
                map.y *= qa.y;
            }
            float2 out;
            chain(a, j, it, map, in, out);
            *reinterpret_cast<float2*>(&sh.in[2 * lane]) = in;
            if (it.last && !it.dead && a.ds0)
                store2_any(a.ds0, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, out.x, out.y);
        }
        // while the chain goes on: the state entering the thread's span, and the gradients' map after it
        float h[4], pa[4] = {1.f, 1.f, 1.f, 1.f}, pc[4] = {0.f, 0.f, 0.f, 0.f};
        get4(&sh.h0[c4], h);
        for (int i = 0; i < w; ++i) {
            float qa[4], qu[4];
            get4(&sh.a[i][c4], qa);
            get4(&sh.u[i][c4], qu);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = fmaf(qa[e], h[e], qu[e]);
        }
        if (half == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = fmaf(oa[e], h[e], ou[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pa[e] = oa[e];
                pc[e] = oc[e];
            }
        }
        for (int i = w + 1; i < kWarps; ++i) {
            float qa[4], qc[4];
            get4(&sh.a[i][c4], qa);
            get4(&sh.c[i][c4], qc);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pc[e] = fmaf(pa[e], qc[e], pc[e]);
                pa[e] *= qa[e];
            }
        }
        __syncthreads();
        if (rows > 0) {
            with_gate(a.mode, a.compl_in, [&](auto gt) {
                constexpr bool kCompl = decltype(gt)::complement, kSlope = decltype(gt)::mode != LA_GATE_LOG;
#pragma unroll 1
                for (int p = 0; p < 4; p += 2) {  // two channels at a time: what a span keeps has to fit the registers
                    float dec[kSpan][2], prev[kSpan][2], m[kSpan][2], slope[kSpan][2];
                    float2 e = *reinterpret_cast<const float2*>(&sh.in[c4 + p]);
                    e.x = fmaf(p ? pa[2] : pa[0], e.x, p ? pc[2] : pc[0]);
                    e.y = fmaf(p ? pa[3] : pa[1], e.y, p ? pc[3] : pc[1]);
                    float h0 = p ? h[2] : h[0], h1 = p ? h[3] : h[1];
#pragma unroll
                    for (int k = 0; k < kSpan; ++k)
                        if (k < n) {
                            const float2 x = get2(wx + mine + k * kChannels + p), g = get2(wg + mine + k * kChannels + p);
                            gate<decltype(gt)::mode, kCompl>(a.lb, g.x, dec[k][0], m[k][0], slope[k][0]);
                            gate<decltype(gt)::mode, kCompl>(a.lb, g.y, dec[k][1], m[k][1], slope[k][1]);
                            prev[k][0] = kCompl ? h0 - x.x : h0;
                            prev[k][1] = kCompl ? h1 - x.y : h1;
                            h0 = fmaf(dec[k][0], h0, kCompl ? m[k][0] * x.x : x.x);
                            h1 = fmaf(dec[k][1], h1, kCompl ? m[k][1] * x.y : x.y);
                        }
#pragma unroll
                    for (int k = kSpan - 1; k >= 0; --k)
                        if (k < n) {
                            const float2 d = get2(wd + mine + k * kChannels + p);
                            e.x += d.x;
                            e.y += d.y;
                            put2(wx + mine + k * kChannels + p, kCompl ? m[k][0] * e.x : e.x, kCompl ? m[k][1] * e.y : e.y);
                            e.x *= dec[k][0];
                            e.y *= dec[k][1];
                            const float g0 = e.x * prev[k][0], g1 = e.y * prev[k][1];
                            put2(wg + mine + k * kChannels + p, kSlope ? g0 * slope[k][0] : g0, kSlope ? g1 * slope[k][1] : g1);
                        }
                }
            });
            if (a.tma && rows == kWarpRows) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tile_store(&maps.out, wx, it.d, it.start + w * kWarpRows);
                    tile_store(&maps.dg, wg, it.d, it.start + w * kWarpRows);
                    bulk_commit_group();
                    bulk_wait_read_all();
                }
            } else {
                __syncwarp();
                rows_out(wx, a.dx, a.dx_st, it.start + w * kWarpRows, rows, it.d, a.D);
                rows_out(wg, a.dg, a.dg_st, it.start + w * kWarpRows, rows, it.d, a.D);
            }
        }
        if (jn >= a.items) break;
        fence_proxy_async_smem();  // the rows were written here, and are about to be by TMA
        __syncwarp();
        fetch(sh.items[at ^ 1]);
        j = jn;
    }
    if (lane == 0) bulk_wait_all();
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) glr_decode_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.N || d >= a.D) return;
    int64_t slot = i;
    if (a.idx) {
        slot = a.idx[i];
        if (slot < 0 || slot >= a.pool) {
            raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
            return;
        }
    }
    float dec, m, slope;
    const float g = to_f(static_cast<const G*>(a.g)[i * a.g_st + d]);
    with_gate(a.mode, a.compl_in, [&](auto gt) { gate<decltype(gt)::mode, decltype(gt)::complement>(a.lb, g, dec, m, slope); });
    const float h = fmaf(dec, load_any(a.s0, slot * a.D + d, a.s0_bf16), m * to_f(static_cast<const X*>(a.x)[i * a.x_st + d]));
    store_any(const_cast<void*>(a.s0), slot * a.D + d, a.s0_bf16, h);
    static_cast<X*>(a.h)[i * a.h_st + d] = from_f<X>(h);
}

template <typename K>
la_status launch_scan(K kernel, size_t smem, Args& a, Maps& maps, cudaStream_t s) {
    int dev = 0, sms = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kScanThreads, smem) != cudaSuccess || per_sm < 1) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.items, static_cast<int64_t>(sms) * per_sm));
    void* args[] = {&a, &maps};
    if (cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(kScanThreads), args, smem, s) != cudaSuccess) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    return LA_OK;
}

enum Which { kFwd, kBwd };

template <typename X, typename G>
la_status scan(Args& a, Maps& maps, Which w, cudaStream_t s) {
    return w == kFwd ? launch_scan(glr_fwd_kernel<X, G>, stage_bytes<X, G, 1>(), a, maps, s)
                     : launch_scan(glr_bwd_kernel<X, G>, stage_bytes<X, G, 2>(), a, maps, s);
}

// The chain's table: maps and states of every item.  None when no sequence can have two blocks.
size_t map_bytes(int64_t T, int32_t N, int32_t D) {
    if (T <= kBlock) return 0;
    return static_cast<size_t>(T / kBlock + N) * ((D + kChannels - 1) / kChannels) * 32 * sizeof(ulonglong2);
}
size_t table_bytes(int64_t T, int32_t N, int32_t D) { return map_bytes(T, N, D) / 2 * 3; }  // a state is half a map

la_status run_scan(Args& a, int32_t xd, int32_t gd, Which w, void* ws, cudaStream_t s) {
    if (a.N == 0) return LA_OK;
    a.tiles = (a.D + kChannels - 1) / kChannels;
    a.items = (a.T / kBlock + a.N) * a.tiles;
    if (a.items >= (int64_t(1) << 31)) return LA_ERR_UNSUPPORTED;
    if (const size_t maps = map_bytes(a.T, a.N, a.D)) {
        a.maps = static_cast<ulonglong2*>(ws);
        a.states = reinterpret_cast<uint2*>(static_cast<uint8_t*>(ws) + maps);
        if (cudaMemsetAsync(ws, 0xFF, table_bytes(a.T, a.N, a.D), s) != cudaSuccess) return LA_ERR_CUDA;
    }
    Maps maps = {};
    auto tile = [&](CUtensorMap* m, const void* p, int64_t stride, int32_t dtype) {
        return tileable(p, stride, a.T, a.D, dtype) && tile_map(m, p, stride, a.T, a.D, dtype, kChannels, kWarpRows);
    };
    a.tma = tile(&maps.x, a.x, a.x_st, xd) && tile(&maps.g, a.g, a.g_st, gd);
    if (w == kFwd) a.tma = a.tma && (!a.h || tile(&maps.out, a.h, a.h_st, xd));
    else a.tma = a.tma && tile(&maps.dh, a.dh, a.dh_st, xd) && tile(&maps.out, a.dx, a.dx_st, xd) && tile(&maps.dg, a.dg, a.dg_st, gd);
    if (xd == LA_DTYPE_BF16) return gd == LA_DTYPE_BF16 ? scan<bf16, bf16>(a, maps, w, s) : scan<bf16, float>(a, maps, w, s);
    return gd == LA_DTYPE_BF16 ? scan<float, bf16>(a, maps, w, s) : scan<float, float>(a, maps, w, s);
}

template <typename X, typename G>
la_status launch_decode(const Args& a, cudaStream_t s) {
    const unsigned ny = std::min(a.N, 65535), nz = (a.N + ny - 1) / ny;
    glr_decode_kernel<X, G><<<dim3((a.D + kThreads - 1) / kThreads, ny, nz), kThreads, 0, s>>>(a);
    return launched();
}

}  // namespace

extern "C" {

size_t la_glr_checkpoint_rows(int64_t T, int32_t N) {
    return T < 0 || N < 0 ? 0 : static_cast<size_t>(T / kBlock + N);
}

size_t la_glr_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t backward, int32_t checkpoints_given) {
    if (T < 0 || N < 0 || D <= 0) return 0;
    const size_t states = backward && !checkpoints_given ? (la_glr_checkpoint_rows(T, N) * D * 4 + 255) & ~size_t(255) : 0;
    return states + table_bytes(T, N, D);
}

la_status glr_fwd(const la_glr_fwd_params* p, void* stream) {
    if (!p || p->D <= 0) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->g_dtype)) return LA_ERR_UNSUPPORTED;
    if (p->initial_state && !known_dtype(p->initial_state_dtype)) return LA_ERR_UNSUPPORTED;
    if ((st = check_gate(p->gate_mode, p->gate_lower_bound)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->g, p->g_stride_t, p->T, p->D, p->g_dtype, false) ||
        !good_rows(p->h, p->h_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_optional(p->initial_state, p->initial_state_dtype) || !good_optional(p->final_state, LA_DTYPE_F32) ||
        !good_optional(p->checkpoints, LA_DTYPE_F32))
        return LA_ERR_INVALID_ARG;
    if (p->state_indices && (!aligned_to(p->state_indices, 4) || !p->initial_state || p->final_state || p->state_pool_size <= 0))
        return LA_ERR_INVALID_ARG;
    if ((st = check_workspace(p->workspace, p->workspace_bytes, la_glr_workspace_bytes(p->T, p->N, p->D, 0, 0))) != LA_OK) return st;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.g = p->g; a.g_st = p->g_stride_t;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D;
    a.mode = p->gate_mode; a.lb = p->gate_lower_bound; a.compl_in = p->complement_input != 0;
    a.s0 = p->initial_state; a.s0_bf16 = p->initial_state_dtype == LA_DTYPE_BF16;
    a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.h = p->h; a.h_st = p->h_stride_t; a.fin = p->final_state; a.ckpt = p->checkpoints;
    a.status = p->status;
    return run_scan(a, p->x_dtype, p->g_dtype, kFwd, p->workspace, static_cast<cudaStream_t>(stream));
}

la_status glr_bwd(const la_glr_bwd_params* p, void* stream) {
    if (!p || p->D <= 0) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->g_dtype)) return LA_ERR_UNSUPPORTED;
    if (p->initial_state && !known_dtype(p->initial_state_dtype)) return LA_ERR_UNSUPPORTED;
    if ((st = check_gate(p->gate_mode, p->gate_lower_bound)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->g, p->g_stride_t, p->T, p->D, p->g_dtype, false) ||
        !good_rows(p->d_h, p->d_h_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->dx, p->dx_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_rows(p->dg, p->dg_stride_t, p->T, p->D, p->g_dtype, true) ||
        !good_optional(p->initial_state, p->initial_state_dtype) || !good_optional(p->checkpoints, LA_DTYPE_F32) ||
        !good_optional(p->d_final_state, LA_DTYPE_F32) || !good_optional(p->d_initial_state, LA_DTYPE_F32))
        return LA_ERR_INVALID_ARG;
    const size_t need = la_glr_workspace_bytes(p->T, p->N, p->D, 1, p->checkpoints != nullptr);
    if ((st = check_workspace(p->workspace, p->workspace_bytes, need)) != LA_OK) return st;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.g = p->g; a.g_st = p->g_stride_t;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D;
    a.mode = p->gate_mode; a.lb = p->gate_lower_bound; a.compl_in = p->complement_input != 0;
    a.s0 = p->initial_state; a.s0_bf16 = p->initial_state_dtype == LA_DTYPE_BF16;
    a.dh = p->d_h; a.dh_st = p->d_h_stride_t; a.dfin = p->d_final_state;
    a.dx = p->dx; a.dx_st = p->dx_stride_t; a.dg = p->dg; a.dg_st = p->dg_stride_t; a.ds0 = p->d_initial_state;
    a.status = p->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.ckpt = const_cast<float*>(p->checkpoints);
    if (!a.ckpt && a.N > 0) {  // the forward again, for the states entering every block, which come after the table
        Args f = a;
        f.ckpt = a.ckpt = reinterpret_cast<float*>(static_cast<uint8_t*>(p->workspace) + table_bytes(a.T, a.N, a.D));
        if ((st = run_scan(f, p->x_dtype, p->g_dtype, kFwd, p->workspace, s)) != LA_OK) return st;
    }
    return run_scan(a, p->x_dtype, p->g_dtype, kBwd, p->workspace, s);
}

la_status glr_decode(const la_glr_decode_params* p, void* stream) {
    if (!p || p->D <= 0 || p->N < 0) return LA_ERR_INVALID_ARG;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->g_dtype) || !known_dtype(p->state_dtype)) return LA_ERR_UNSUPPORTED;
    la_status st = check_gate(p->gate_mode, p->gate_lower_bound);
    if (st != LA_OK) return st;
    if (!p->state_pool || !good_optional(p->state_pool, p->state_dtype) || p->state_pool_size <= 0) return LA_ERR_INVALID_ARG;
    if (p->state_indices ? !aligned_to(p->state_indices, 4) : p->state_pool_size < p->N) return LA_ERR_INVALID_ARG;
    if (!good_rows(p->x, p->x_stride_n, p->N, p->D, p->x_dtype, false) ||
        !good_rows(p->g, p->g_stride_n, p->N, p->D, p->g_dtype, false) ||
        !good_rows(p->h, p->h_stride_n, p->N, p->D, p->x_dtype, true))
        return LA_ERR_INVALID_ARG;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_n; a.g = p->g; a.g_st = p->g_stride_n;
    a.N = p->N; a.D = p->D;
    a.mode = p->gate_mode; a.lb = p->gate_lower_bound; a.compl_in = p->complement_input != 0;
    a.s0 = p->state_pool; a.s0_bf16 = p->state_dtype == LA_DTYPE_BF16;
    a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.h = p->h; a.h_st = p->h_stride_n;
    a.status = p->status;
    if (a.N == 0) return LA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->x_dtype == LA_DTYPE_BF16) return p->g_dtype == LA_DTYPE_BF16 ? launch_decode<bf16, bf16>(a, s) : launch_decode<bf16, float>(a, s);
    return p->g_dtype == LA_DTYPE_BF16 ? launch_decode<float, bf16>(a, s) : launch_decode<float, float>(a, s);
}

}  // extern "C"
