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
// a block of 128 tokens x 64 channels into registers (each thread 8 tokens of 2 channels), composes
// its warps' maps in shared memory, and needs one number per channel from the block before: the
// state entering it.  That chain runs through a table in the workspace.  A block publishes its
// composed map (A, B) as soon as it has it and the state leaving it once it knows the one entering;
// a block that needs a state looks back over up to 32 predecessors, takes the nearest published
// state and folds the maps after it in order.  The state leaving a block is always
// fma(A, entering, B), whoever computes it, so the bits do not depend on what was published when.
// The launch is cooperative (all CTAs resident), every CTA walks its items in ascending order and
// items only wait for lower ones, so the lowest unfinished item never waits and the waits end; they
// are bounded all the same.  Each operand is read once and each result written once.
//
// The backward runs the same chain from each sequence's end, over the gradient leaving a token,
// c_t = a_t (dh_t + c_{t+1}); the states entering its blocks come from the forward's checkpoints (one
// row per 128 tokens, 1.5 % of the operands' bytes), so it is one pass too.
#include <algorithm>

#include "mixer.cuh"

namespace {

using namespace la::mixer;

constexpr int kThreads = 128;                          // decode
constexpr int kSpan = 8;                               // tokens of a thread
constexpr int kWarps = 16;                             // of a CTA, one span each
constexpr int kScanThreads = 32 * kWarps;
constexpr int kBlock = kSpan * kWarps;                 // tokens of a block, and between saved states
constexpr int kChannels = 64;                          // of a CTA, two a lane
constexpr uint64_t kWaitNs = 1000000000ull;            // a bounded wait gives up after a second
static_assert(kBlock == 128, "the checkpoint cadence of the interface");

// a, m and dl/dg of one gate value.  The log sigmoid's a = s(g) and 1 - a = s(-g) come from
// e = exp(-|g|) without cancellation; otherwise 1 - a = -expm1(l).
__device__ __forceinline__ void gate(int mode, float lb, bool compl_in, float g, float& a, float& m, float& slope) {
    if (mode == LA_GATE_LOGSIGMOID) {
        const float e = expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
        a = g >= 0.f ? big : small;
        slope = g >= 0.f ? small : big;
        m = compl_in ? slope : 1.f;
        return;
    }
    float l = g;
    slope = 1.f;
    if (mode == LA_GATE_SIGMOID_BOUND) {
        const float e = expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
        l = lb * (g >= 0.f ? big : small);
        slope = l * (g >= 0.f ? small : big);
    }
    a = expf(l);
    m = compl_in ? -expm1f(l) : 1.f;
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
};

// ---------------------------------------------------------------- asynchronous copies
// One thread's two channels of one token (4 or 8 bytes) into its own place in shared memory.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <typename T>
struct Pair {
    T v[2];
};

// The channels d, d + 1 of one row; kPair: as one 2-element access (D even, everything aligned).
template <typename T, bool kPair>
__device__ __forceinline__ void load2(const void* base, int64_t at, int d, int D, float& v0, float& v1) {
    const T* p = static_cast<const T*>(base) + at + d;
    if (kPair) {
        if (sizeof(T) == 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
            v0 = __uint_as_float(w << 16);
            v1 = __uint_as_float(w & 0xFFFF0000u);
        } else {
            const float2 w = *reinterpret_cast<const float2*>(p);
            v0 = w.x;
            v1 = w.y;
        }
    } else {
        v0 = to_f(p[0]);
        v1 = d + 1 < D ? to_f(p[1]) : 0.f;
    }
}
template <typename T, bool kPair>
__device__ __forceinline__ void store2(void* base, int64_t at, int d, int D, float v0, float v1) {
    T* p = static_cast<T*>(base) + at + d;
    if (kPair) {
        if (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v0, v1);
        else *reinterpret_cast<float2*>(p) = make_float2(v0, v1);
    } else {
        p[0] = from_f<T>(v0);
        if (d + 1 < D) p[1] = from_f<T>(v1);
    }
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

// Shared memory: one staging place per thread, token and operand, then the warps' maps.
template <typename X, typename G, int kX>
constexpr size_t stage_bytes() { return static_cast<size_t>(kScanThreads) * kSpan * (kX * sizeof(Pair<X>) + sizeof(Pair<G>)); }

template <typename X, typename G, bool kPair>
__global__ void __launch_bounds__(kScanThreads, 2) glr_fwd_kernel(const Args a) {
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ float4 maps[kWarps][32];
    __shared__ float2 enter[kWarps][32];
    Pair<X>* sx = reinterpret_cast<Pair<X>*>(stage) + threadIdx.x;
    Pair<G>* sg = reinterpret_cast<Pair<G>*>(stage + static_cast<size_t>(kScanThreads) * kSpan * sizeof(Pair<X>)) + threadIdx.x;
    __shared__ Item items[2];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    check_boundaries(a);

    auto fetch = [&](const Item& it) {
        const int d = it.d + 2 * lane, n = d < a.D ? it.count - w * kSpan : 0;
        const int64_t t = it.start + w * kSpan;
#pragma unroll
        for (int k = 0; k < kSpan; ++k)
            if (k < n) {
                copy_async<sizeof(Pair<X>)>(sx + k * kScanThreads, static_cast<const X*>(a.x) + (t + k) * a.x_st + d);
                copy_async<sizeof(Pair<G>)>(sg + k * kScanThreads, static_cast<const G*>(a.g) + (t + k) * a.g_st + d);
            }
        copies_commit();
    };

    int64_t j = blockIdx.x;
    if (w == 0) locate<false>(a, j, &items[0]);
    __syncthreads();
    if (kPair) fetch(items[0]);
    for (int at = 0;; at ^= 1) {
        const Item& it = items[at];
        const int64_t jn = j + gridDim.x;
        // the next item, while this one's operands arrive; nobody reads its place any more
        if (w == kWarps - 1 && jn < a.items) locate<false>(a, jn, &items[at ^ 1]);
        const int ch = it.d + 2 * lane;  // this lane's first channel
        const int n = ch < a.D ? it.count - w * kSpan : 0;
        const int64_t t = it.start + w * kSpan;
        float dec[kSpan][2], u[kSpan][2];
        if (kPair) copies_wait();
        float4 map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSpan; ++k) {
            dec[k][0] = dec[k][1] = 1.f;
            u[k][0] = u[k][1] = 0.f;
            if (k < n) {
                float x0, x1, g0, g1, m0, m1, slope;
                if (kPair) {
                    load2<X, true>(sx + k * kScanThreads, 0, 0, 2, x0, x1);
                    load2<G, true>(sg + k * kScanThreads, 0, 0, 2, g0, g1);
                } else {
                    load2<X, false>(a.x, (t + k) * a.x_st, ch, a.D, x0, x1);
                    load2<G, false>(a.g, (t + k) * a.g_st, ch, a.D, g0, g1);
                }
                gate(a.mode, a.lb, a.compl_in, g0, dec[k][0], m0, slope);
                gate(a.mode, a.lb, a.compl_in, g1, dec[k][1], m1, slope);
                u[k][0] = m0 * x0;
                u[k][1] = m1 * x1;
                map.z = fmaf(dec[k][0], map.z, u[k][0]);
                map.w = fmaf(dec[k][1], map.w, u[k][1]);
                map.x *= dec[k][0];
                map.y *= dec[k][1];
            }
        }
        maps[w][lane] = map;
        __syncthreads();
        if (kPair && jn < a.items) fetch(items[at ^ 1]);
        if (w == 0) {
            float2 in = make_float2(0.f, 0.f), out = in;
            if (it.order == 0 && !it.dead && a.s0) load2_any(a.s0, it.state * static_cast<int64_t>(a.D), ch, a.D, a.s0_bf16, in.x, in.y);
            map = maps[0][lane];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                const float4 q = maps[i][lane];
                map.z = fmaf(q.x, map.z, q.z);
                map.w = fmaf(q.y, map.w, q.w);
                map.x *= q.x;
                map.y *= q.y;
            }
            chain(a, j, it, map, in, out);
            if (!it.dead) {
                if (a.ckpt && it.count > 0) store2_any(a.ckpt, it.slot * static_cast<int64_t>(a.D), ch, a.D, 0, in.x, in.y);
                if (it.last) {
                    if (a.idx) store2_any(const_cast<void*>(a.s0), it.state * static_cast<int64_t>(a.D), ch, a.D, a.s0_bf16, out.x, out.y);
                    else if (a.fin) store2_any(a.fin, it.state * static_cast<int64_t>(a.D), ch, a.D, 0, out.x, out.y);
                }
            }
            enter[0][lane] = in;
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                const float4 q = maps[i - 1][lane];
                in.x = fmaf(q.x, in.x, q.z);
                in.y = fmaf(q.y, in.y, q.w);
                enter[i][lane] = in;
            }
        }
        __syncthreads();
        if (a.h) {
            float2 h = enter[w][lane];
#pragma unroll
            for (int k = 0; k < kSpan; ++k)
                if (k < n) {
                    h.x = fmaf(dec[k][0], h.x, u[k][0]);
                    h.y = fmaf(dec[k][1], h.y, u[k][1]);
                    store2<X, kPair>(a.h, (t + k) * a.h_st, ch, a.D, h.x, h.y);
                }
        }
        if (jn >= a.items) break;
        j = jn;
    }
}

// kPlain: log decay without the complement, where m = dl/dg = 1.
template <typename X, typename G, bool kPair, bool kPlain>
__global__ void __launch_bounds__(kScanThreads, 1) glr_bwd_kernel(const Args a) {
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ float4 maps[kWarps][32];   // (a, a, u, u) of the states
    __shared__ float2 grads[kWarps][32];  // the constant part of the gradients' map
    __shared__ float2 enter[kWarps][32], leave[kWarps][32];
    constexpr size_t kPlane = static_cast<size_t>(kScanThreads) * kSpan;
    Pair<X>* sx = reinterpret_cast<Pair<X>*>(stage) + threadIdx.x;
    Pair<X>* sd = sx + kPlane;
    Pair<G>* sg = reinterpret_cast<Pair<G>*>(stage + 2 * kPlane * sizeof(Pair<X>)) + threadIdx.x;
    __shared__ Item items[2];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    check_boundaries(a);

    auto fetch = [&](const Item& it) {
        const int d = it.d + 2 * lane, n = d < a.D ? it.count - w * kSpan : 0;
        const int64_t t = it.start + w * kSpan;
#pragma unroll
        for (int k = 0; k < kSpan; ++k)
            if (k < n) {
                copy_async<sizeof(Pair<X>)>(sx + k * kScanThreads, static_cast<const X*>(a.x) + (t + k) * a.x_st + d);
                copy_async<sizeof(Pair<X>)>(sd + k * kScanThreads, static_cast<const X*>(a.dh) + (t + k) * a.dh_st + d);
                copy_async<sizeof(Pair<G>)>(sg + k * kScanThreads, static_cast<const G*>(a.g) + (t + k) * a.g_st + d);
            }
        copies_commit();
    };

    int64_t j = blockIdx.x;
    if (w == 0) locate<true>(a, j, &items[0]);
    __syncthreads();
    if (kPair) fetch(items[0]);
    for (int at = 0;; at ^= 1) {
        const Item& it = items[at];
        const int64_t jn = j + gridDim.x;
        // the next item, while this one's operands arrive; nobody reads its place any more
        if (w == kWarps - 1 && jn < a.items) locate<true>(a, jn, &items[at ^ 1]);
        const int ch = it.d + 2 * lane;  // this lane's first channel
        const int n = ch < a.D ? it.count - w * kSpan : 0;
        const int64_t t = it.start + w * kSpan;
        float dec[kSpan][2], u[kSpan][2], d[kSpan][2], x[kSpan][2], m[kSpan][2], slope[kSpan][2];
        if (kPair) copies_wait();
        float4 map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSpan; ++k) {
            dec[k][0] = dec[k][1] = 1.f;
            u[k][0] = u[k][1] = d[k][0] = d[k][1] = 0.f;
            if (k < n) {
                float g0, g1;
                if (kPair) {
                    load2<X, true>(sx + k * kScanThreads, 0, 0, 2, x[k][0], x[k][1]);
                    load2<X, true>(sd + k * kScanThreads, 0, 0, 2, d[k][0], d[k][1]);
                    load2<G, true>(sg + k * kScanThreads, 0, 0, 2, g0, g1);
                } else {
                    load2<X, false>(a.x, (t + k) * a.x_st, ch, a.D, x[k][0], x[k][1]);
                    load2<X, false>(a.dh, (t + k) * a.dh_st, ch, a.D, d[k][0], d[k][1]);
                    load2<G, false>(a.g, (t + k) * a.g_st, ch, a.D, g0, g1);
                }
                if (kPlain) {
                    dec[k][0] = expf(g0);
                    dec[k][1] = expf(g1);
                    u[k][0] = x[k][0];
                    u[k][1] = x[k][1];
                } else {
                    gate(a.mode, a.lb, a.compl_in, g0, dec[k][0], m[k][0], slope[k][0]);
                    gate(a.mode, a.lb, a.compl_in, g1, dec[k][1], m[k][1], slope[k][1]);
                    u[k][0] = m[k][0] * x[k][0];
                    u[k][1] = m[k][1] * x[k][1];
                }
                map.z = fmaf(dec[k][0], map.z, u[k][0]);
                map.w = fmaf(dec[k][1], map.w, u[k][1]);
                map.x *= dec[k][0];
                map.y *= dec[k][1];
            }
        }
        float2 c = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = kSpan - 1; k >= 0; --k) {
            c.x = dec[k][0] * (d[k][0] + c.x);
            c.y = dec[k][1] * (d[k][1] + c.y);
        }
        maps[w][lane] = map;
        grads[w][lane] = c;
        __syncthreads();
        if (kPair && jn < a.items) fetch(items[at ^ 1]);
        if (w == 0) {
            float2 in = make_float2(0.f, 0.f), out = in;
            if (it.order == 0 && !it.dead && a.dfin) load2_any(a.dfin, it.state * static_cast<int64_t>(a.D), ch, a.D, 0, in.x, in.y);
            map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
            for (int i = kWarps - 1; i >= 0; --i) {
                const float4 q = maps[i][lane];
                const float2 e = grads[i][lane];
                map.z = fmaf(q.x, map.z, e.x);
                map.w = fmaf(q.y, map.w, e.y);
                map.x *= q.x;
                map.y *= q.y;
            }
            chain(a, j, it, map, in, out);
            if (it.last && !it.dead && a.ds0) store2_any(a.ds0, it.state * static_cast<int64_t>(a.D), ch, a.D, 0, out.x, out.y);
#pragma unroll
            for (int i = kWarps - 1; i >= 0; --i) {
                leave[i][lane] = in;
                const float4 q = maps[i][lane];
                const float2 e = grads[i][lane];
                in.x = fmaf(q.x, in.x, e.x);
                in.y = fmaf(q.y, in.y, e.y);
            }
        } else if (w == 1) {
            float2 h = make_float2(0.f, 0.f);
            if (it.count > 0) load2_any(a.ckpt, it.slot * static_cast<int64_t>(a.D), ch, a.D, 0, h.x, h.y);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                enter[i][lane] = h;
                const float4 q = maps[i][lane];
                h.x = fmaf(q.x, h.x, q.z);
                h.y = fmaf(q.y, h.y, q.w);
            }
        }
        __syncthreads();
        float2 h = enter[w][lane];
#pragma unroll
        for (int k = 0; k < kSpan; ++k) {  // u becomes h_{t-1}
            const float u0 = u[k][0], u1 = u[k][1];
            u[k][0] = h.x;
            u[k][1] = h.y;
            h.x = fmaf(dec[k][0], h.x, u0);
            h.y = fmaf(dec[k][1], h.y, u1);
        }
        float2 e = leave[w][lane];
#pragma unroll
        for (int k = kSpan - 1; k >= 0; --k) {
            if (k >= n) continue;
            e.x += d[k][0];
            e.y += d[k][1];
            if (kPlain) store2<X, kPair>(a.dx, (t + k) * a.dx_st, ch, a.D, e.x, e.y);
            else store2<X, kPair>(a.dx, (t + k) * a.dx_st, ch, a.D, m[k][0] * e.x, m[k][1] * e.y);
            e.x *= dec[k][0];
            e.y *= dec[k][1];
            if (kPlain) {
                store2<G, kPair>(a.dg, (t + k) * a.dg_st, ch, a.D, e.x * u[k][0], e.y * u[k][1]);
            } else {
                const float p0 = a.compl_in ? u[k][0] - x[k][0] : u[k][0], p1 = a.compl_in ? u[k][1] - x[k][1] : u[k][1];
                store2<G, kPair>(a.dg, (t + k) * a.dg_st, ch, a.D, e.x * p0 * slope[k][0], e.y * p1 * slope[k][1]);
            }
        }
        if (jn >= a.items) break;
        j = jn;
    }
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
    gate(a.mode, a.lb, a.compl_in, to_f(static_cast<const G*>(a.g)[i * a.g_st + d]), dec, m, slope);
    const float h = fmaf(dec, load_any(a.s0, slot * a.D + d, a.s0_bf16), m * to_f(static_cast<const X*>(a.x)[i * a.x_st + d]));
    store_any(const_cast<void*>(a.s0), slot * a.D + d, a.s0_bf16, h);
    static_cast<X*>(a.h)[i * a.h_st + d] = from_f<X>(h);
}

template <typename K>
la_status launch_scan(K kernel, size_t smem, Args& a, cudaStream_t s) {
    int dev = 0, sms = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kScanThreads, smem) != cudaSuccess || per_sm < 1) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.items, static_cast<int64_t>(sms) * per_sm));
    void* args[] = {&a};
    if (cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(kScanThreads), args, smem, s) != cudaSuccess) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    return LA_OK;
}

// Whether every row of the operand starts on a boundary of two of its elements.
bool pairs(const void* p, int64_t stride, int64_t T, int32_t dtype) {
    return aligned_to(p, 2 * dtype_size(dtype)) && (T == 1 || stride % 2 == 0);
}

enum Which { kFwd, kBwd };

template <typename X, typename G>
la_status scan(Args& a, Which w, bool pair, cudaStream_t s) {
    if (w == kFwd) {
        const size_t smem = pair ? stage_bytes<X, G, 1>() : 0;
        return pair ? launch_scan(glr_fwd_kernel<X, G, true>, smem, a, s) : launch_scan(glr_fwd_kernel<X, G, false>, smem, a, s);
    }
    const size_t smem = pair ? stage_bytes<X, G, 2>() : 0;
    const bool plain = a.mode == LA_GATE_LOG && !a.compl_in;
    if (pair) return plain ? launch_scan(glr_bwd_kernel<X, G, true, true>, smem, a, s) : launch_scan(glr_bwd_kernel<X, G, true, false>, smem, a, s);
    return plain ? launch_scan(glr_bwd_kernel<X, G, false, true>, smem, a, s) : launch_scan(glr_bwd_kernel<X, G, false, false>, smem, a, s);
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
    bool pair = a.D % 2 == 0 && pairs(a.x, a.x_st, a.T, xd) && pairs(a.g, a.g_st, a.T, gd);
    if (w == kFwd) pair = pair && (!a.h || pairs(a.h, a.h_st, a.T, xd));
    else pair = pair && pairs(a.dh, a.dh_st, a.T, xd) && pairs(a.dx, a.dx_st, a.T, xd) && pairs(a.dg, a.dg_st, a.T, gd);
    if (xd == LA_DTYPE_BF16) return gd == LA_DTYPE_BF16 ? scan<bf16, bf16>(a, w, pair, s) : scan<bf16, float>(a, w, pair, s);
    return gd == LA_DTYPE_BF16 ? scan<float, bf16>(a, w, pair, s) : scan<float, float>(a, w, pair, s);
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
