// ssm.cuh -- the selective state space scan (ssm_fwd, ssm_bwd, ssm_decode): what ssm_fwd.cu, ssm_bwd.cu and ssm.cu share.
//
// Channel d of group j, states s, with the step size dt_t (the raw one plus the bias, through softplus where asked for):
//
//   a_t = e^(dt_t A[d, s]),  h_t = a_t h_{t-1} + dt_t x_t B_t[j, s],  p_t = sum_s C_t[j, s] h_t + skip[d] x_t,
//   y_t = p_t  or  p_t silu(z_t);
//
// and backwards, dp being the gradient of p and g_t the one that leaves token t towards h_{t-1}:
//
//   e_t = C_t dp_t + g_{t+1},  g_t = a_t e_t,  dC_t = sum_d dp h_t,  dB_t = sum_d e_t dt x,  du = sum_s e_t B_t,
//   w_t = g_t h_{t-1},  dA += w_t dt,  dx = du dt + dp skip,  d dt = du x + sum_s w_t A.
//
// States stay in registers while a lane walks the tokens; the ones beyond S (up to 64) have A = B = C = 0.  In the scan, the
// gradient behind each block and the small batches' single tokens a lane has 8 or 16 states of one channel, which Q = 1, 2 or 4
// lanes share.  In the kernel of all gradients it has four states of four channels (Q = 4, 8 or 16 lanes share them), for the large
// batches' single tokens four states of one channel (Q = 1 to 16).
#pragma once
#include <algorithm>

#include "mixer.cuh"

namespace la {
namespace ssm {

using namespace la::mixer;

constexpr int kSave = 16;  // tokens between saved states
constexpr int kMaxS = 64;
constexpr int kSms = 152;

// A decay is ex2(dt (A log2(e)) + kEx2Low), the same bits in the scans and for single tokens.  ex2.approx is low on average just
// below 1, where an error adds up over 1 / |dt A| tokens: by 0.10 to 0.13 units of 2^-24 for |dt A| of 1e-5 to 1e-3, by 0.25 to
// 0.35 from there to 1/2 (measured over 4e6 decays each).  0.22 in its argument leaves means within 0.13 throughout.
constexpr float kEx2Low = 0.22f * 0x1p-24f * kLog2e;

struct Args {
    const void *x, *dt, *z, *b, *c, *dy;
    int64_t x_st, dt_st, z_st, dy_st, b_st, b_sg, c_st, c_sg;
    const float *A, *skip, *bias;
    int softplus;
    const void* cu;
    int cu64, N;
    int64_t T;
    int D, S, G, Dg, tiles_pg;  // channels and channel tiles of a group
    const void* s0;
    int s0_bf16;
    const int32_t* idx;
    int64_t pool;
    void* y;
    int64_t y_st;
    float *fin, *ckpt;
    const float* dfin;
    void *dx, *ddt, *dz, *db, *dc;
    int64_t dx_st, ddt_st, dz_st;
    float *dA, *dskip, *dbias, *ds0;
    int32_t* status;
    int shift;           // a time block is 2^shift tokens
    float *table, *sums; // [blocks][D][S]: what a block leaves from nothing, then what enters it; [blocks][D]: its steps' sum
    float* dbc;          // [tiles of a group][T][G][2][S]: dB and dC of a tile's channels
    float *pA, *pch;     // [parts][D][S], [parts][2][D]: partial sums of dA, and of d skip and d bias
    int parts;
    int vec, svec;       // wide accesses: rows of the operands; of the states
};

// ---------------------------------------------------------------- time blocks of 2^shift tokens
// Blocks start at each sequence's first token.  Two numberings, both of (T >> shift) + N blocks and found without a table:
// slots, block c of sequence i being (cu[i] >> shift) + i + c (seq_search.h), the rows of the saved states; and launch order,
// the first blocks of all sequences before all others, block c > 0 of sequence i being N + (cu[i] >> shift) + c - 1 (a
// sequence of L tokens has (L - 1) >> shift of those, and no more fit between its boundaries' quotients).
LA_HOST_DEVICE int64_t slots_for(int64_t T, int32_t N, int shift) { return (T >> shift) + N; }

__device__ __forceinline__ SeqBlock time_block(const Args& a, int shift, int32_t seq, int64_t s0, int64_t s1, int64_t c) {
    SeqBlock b;
    b.seq = -1;
    b.start = b.count = b.c = b.len = b.first = 0;
    if (s0 < 0 || s1 < s0 || s1 > a.T || c < 0 || (c > 0 && (c << shift) >= s1 - s0)) return b;
    b.seq = seq;
    b.c = static_cast<int32_t>(c);
    b.first = static_cast<int32_t>(s0);
    b.len = static_cast<int32_t>(s1 - s0);
    b.start = static_cast<int32_t>(s0 + (c << shift));
    b.count = static_cast<int32_t>(min(s1 - b.start, int64_t(1) << shift));
    return b;
}
// The last sequence i whose number (cu[i] >> shift) + i kOwn is at or before `at`; called by whole warps.
template <int kOwn>
__device__ __forceinline__ int32_t find_sequence(const Args& a, int shift, int64_t at) {
    const int lane = threadIdx.x & 31;
    SlotSearch f = {0, a.N, true};
    while (f.n > 1) {
        const int32_t i = f.lo + lane * f.step();
        const bool live = lane * f.step() < f.n;
        const int64_t v = live ? (cu_load(a.cu, a.cu64, i) >> shift) + i * kOwn : 0;
        const unsigned here = __ballot_sync(0xffffffffu, live && v <= at);
        f.narrow(here, here);
    }
    return f.lo;
}
__device__ __forceinline__ SeqBlock find_slot(const Args& a, int shift, int64_t slot) {
    const int32_t i = find_sequence<1>(a, shift, slot);
    const int64_t s0 = cu_load(a.cu, a.cu64, i), s1 = cu_load(a.cu, a.cu64, i + 1);
    return time_block(a, shift, i, s0, s1, slot - ((s0 >> shift) + i));
}
// Sequences of up to two blocks stay whole.
LA_HOST_DEVICE bool split(int64_t len, int shift) { return len > int64_t(2) << shift; }
__device__ __forceinline__ SeqBlock find_launched(const Args& a, int shift, int64_t n) {
    const bool first = n < a.N;
    const int32_t i = first ? static_cast<int32_t>(n) : find_sequence<0>(a, shift, n - a.N);
    const int64_t s0 = cu_load(a.cu, a.cu64, i), s1 = cu_load(a.cu, a.cu64, i + 1);
    SeqBlock b = time_block(a, shift, i, s0, s1, first ? 0 : n - a.N - (s0 >> shift) + 1);
    if (b.seq >= 0 && !split(b.len, shift)) {
        if (first) b.count = b.len;
        else b.seq = -1;
    }
    return b;
}
__device__ __forceinline__ int64_t launched_row(const Args& a, int shift, int64_t seq, int64_t first, int64_t c) {
    return c == 0 ? seq : a.N + (first >> shift) + c - 1;
}
__device__ __forceinline__ int64_t this_slot() { return blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z; }

// Where a sequence's state is in initial_state, or -1 with the status set.
__device__ __forceinline__ int64_t state_row(const Args& a, int32_t seq) {
    if (!a.idx) return seq;
    const int64_t k = a.idx[seq];
    if (k < 0 || k >= a.pool) {
        raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
        return -1;
    }
    return k;
}

// Walks kAhead blocks: each takes the state (or gradient) v that enters it by take(k, v) and leaves e^(its steps' sum a) v + left.
// Rates above 0 may lift the factor beyond the 32-bit range: it then comes in two halves, and a state of 0 stays 0 beside it
// (asked once for all blocks: a branch at each would hold back the next loads, 150 instead of 85 us for 65536 x 2048 x 16 back).
template <int kAhead, typename Take>
__device__ __forceinline__ float walk_blocks(float v, float A2, const float (&sum)[kAhead], const float (&left)[kAhead], Take take) {
    bool grows = false;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) grows |= A2 * sum[k] > 127.f;
    if (grows) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (take(k, v)) {
                const float half = ex2(0.5f * (A2 * sum[k]));
                v = v == 0.f ? left[k] : fmaf(half, half * v, left[k]);
            }
        return v;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (take(k, v)) v = fmaf(ex2(A2 * sum[k]), v, left[k]);
    return v;
}

// ---------------------------------------------------------------- steps
// softplus(v) = max(v, 0) + log1p(t), t = e^-|v| in (0, 1]; log1p(t) = 2 atanh(s), s = t / (2 + t) up to 1/3, where a
// polynomial of degree 4 in s^2 (fitted at Chebyshev nodes) is off by 4e-9: no difference of near values anywhere, and two
// MUFU operations and some ten others where expf and log1pf take forty.
__device__ __forceinline__ float2 softplus2(float2 v) {
    const float2 l = mul2(make_float2(fabsf(v.x), fabsf(v.y)), both(-kLog2e)), t = make_float2(ex2(l.x), ex2(l.y));
    const float2 d = add2(t, both(2.f)), s = mul2(t, make_float2(rcp_fast(d.x), rcp_fast(d.y))), w = mul2(s, s);
    float2 p = fma2(w, both(0.28174657f), both(0.27961419f));
    p = fma2(w, p, both(0.40024854f));
    p = fma2(w, p, both(0.66666316f));
    p = fma2(w, p, both(2.f));
    return fma2(s, p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float2 steps_of(float2 raw, int softplus) { return softplus ? softplus2(raw) : raw; }

// ---------------------------------------------------------------- channels of a tile, lanes of a thread
struct Tile {
    int group, ch, n;  // the tile's group, first channel and number of channels
};
__device__ __forceinline__ Tile tile_of(const Args& a, int tile, int width) {
    Tile t;
    t.group = tile / a.tiles_pg;
    const int at = (tile - t.group * a.tiles_pg) * width;
    t.ch = t.group * a.Dg + at;
    t.n = min(width, a.Dg - at);
    return t;
}

// Four consecutive elements of a row, of which n exist (0 for the others).
template <typename X>
__device__ __forceinline__ float4 load4(const void* base, int64_t at, int n, int vec) {
    const X* p = static_cast<const X*>(base) + at;
    float v[4];
    if (vec && n >= 4) {
        Packed<X, 4> w;
        w.load(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}
template <typename X>
__device__ __forceinline__ void store4(void* base, int64_t at, int n, int vec, float4 f) {
    X* p = static_cast<X*>(base) + at;
    const float v[4] = {f.x, f.y, f.z, f.w};
    if (vec && n >= 4) store_packed<X, 4>(p, v);
    else
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = from_f<X>(v[i]);
}
__device__ __forceinline__ float2 lo(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi(float4 v) { return make_float2(v.z, v.w); }

// ---------------------------------------------------------------- rows into shared memory
__device__ __forceinline__ void cp_async16(void* s, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A thread's part of stages of kTokens rows of n elements, padded with zeros to kWidth in shared memory: the same columns of
// every kRows-th row.
template <typename X, int kWidth, int kThreads, int kTokens>
struct Rows {
    static constexpr int kVec = 16 / static_cast<int>(sizeof(X)), kVecs = kWidth / kVec, kRows = kThreads / kVecs;
    const X* from;  // this thread's column of its first row
    int64_t stride;
    int n;          // elements from this thread's column on
    bool wide;
    __device__ __forceinline__ Rows(const void* base, int64_t at, int64_t stride_, int elements, int vec) : stride(stride_) {
        const int c = threadIdx.x % kThreads % kVecs * kVec;
        n = elements - c;
        wide = vec && n >= kVec;
        from = static_cast<const X*>(base) + at + threadIdx.x % kThreads / kVecs * stride + c;
    }
    // Rows from t on, of which `rows` are left.
    __device__ __forceinline__ void stage(X* to, int t, int rows) const {
        const int i = threadIdx.x % kThreads, r = i / kVecs;
        to += r * kWidth + i % kVecs * kVec;
        const X* p = from + t * stride;
#pragma unroll
        for (int j = 0; j < (kTokens + kRows - 1) / kRows; ++j, to += kRows * kWidth, p += kRows * stride) {
            if (r + j * kRows >= min(rows, kTokens)) continue;
            if (wide) cp_async16(to, p);
            else
#pragma unroll
                for (int e = 0; e < kVec; ++e) to[e] = e < n ? p[e] : from_f<X>(0.f);
        }
    }
};

// Four states of one channel in a [rows, D, S] array; 0 beyond S or where the channel does not exist.
__device__ __forceinline__ float4 load_states(const void* base, int64_t row, const Args& a, int d, int s, bool live, int is_bf16) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (!live || s >= a.S) return make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t at = (row * a.D + d) * a.S + s;
    if (a.svec && !is_bf16) return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    if (a.svec) {
        Packed<bf16, 4> w;
        w.load(static_cast<const bf16*>(base) + at);
        return make_float4(w.get(0), w.get(1), w.get(2), w.get(3));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (s + i < a.S) v[i] = load_any(base, at + i, is_bf16);
    return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_states(void* base, int64_t row, const Args& a, int d, int s, bool live, int is_bf16, float4 f) {
    if (!live || s >= a.S) return;
    const int64_t at = (row * a.D + d) * a.S + s;
    if (a.svec && !is_bf16) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = f;
        return;
    }
    const float v[4] = {f.x, f.y, f.z, f.w};
    if (a.svec) {
        store_packed<bf16, 4>(static_cast<bf16*>(base) + at, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (s + i < a.S) store_any(base, at + i, is_bf16, v[i]);
}

// A thread's kPairs x 2 channels of four states, as pairs of channels: v[p][s] = channels (2p, 2p + 1), state s.
template <int kPairs>
__device__ __forceinline__ void load_thread_states(float2 (&v)[kPairs][4], const void* base, int64_t row, const Args& a, int d, int end, int s, int is_bf16) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        const float4 x = load_states(base, row, a, d + 2 * p, s, d + 2 * p < end, is_bf16);
        const float4 y = load_states(base, row, a, d + 2 * p + 1, s, d + 2 * p + 1 < end, is_bf16);
        v[p][0] = make_float2(x.x, y.x);
        v[p][1] = make_float2(x.y, y.y);
        v[p][2] = make_float2(x.z, y.z);
        v[p][3] = make_float2(x.w, y.w);
    }
}
template <int kPairs>
__device__ __forceinline__ void store_thread_states(const float2 (&v)[kPairs][4], void* base, int64_t row, const Args& a, int d, int end, int s, int is_bf16) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        store_states(base, row, a, d + 2 * p, s, d + 2 * p < end, is_bf16, make_float4(v[p][0].x, v[p][1].x, v[p][2].x, v[p][3].x));
        store_states(base, row, a, d + 2 * p + 1, s, d + 2 * p + 1 < end, is_bf16, make_float4(v[p][0].y, v[p][1].y, v[p][2].y, v[p][3].y));
    }
}
template <int kPairs>
__device__ __forceinline__ void zero(float2 (&v)[kPairs][4]) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s) v[p][s] = both(0.f);
}

// kS consecutive states of a lane's channel, as pairs.
template <int kS>
__device__ __forceinline__ void load_lane_states(float2 (&v)[kS / 2], const void* base, int64_t row, const Args& a, int d, int s, bool live, int is_bf16) {
    if (is_bf16 && a.svec && a.S % 8 == 0) {  // eight at a time
#pragma unroll
        for (int k = 0; k < kS; k += 8) {
            Packed<bf16, 8> w;
            if (live && s + k < a.S) w.load(static_cast<const bf16*>(base) + (row * a.D + d) * a.S + s + k);
            else w.zero();
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k / 2 + i] = make_float2(w.get(2 * i), w.get(2 * i + 1));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kS; k += 4) {
        const float4 f = load_states(base, row, a, d, s + k, live, is_bf16);
        v[k / 2] = lo(f);
        v[k / 2 + 1] = hi(f);
    }
}
template <int kS>
__device__ __forceinline__ void store_lane_states(const float2 (&v)[kS / 2], void* base, int64_t row, const Args& a, int d, int s, bool live, int is_bf16) {
    if (is_bf16 && a.svec && a.S % 8 == 0) {
#pragma unroll
        for (int k = 0; k < kS; k += 8) {
            const float f[8] = {v[k / 2].x, v[k / 2].y, v[k / 2 + 1].x, v[k / 2 + 1].y, v[k / 2 + 2].x, v[k / 2 + 2].y, v[k / 2 + 3].x, v[k / 2 + 3].y};
            if (live && s + k < a.S) store_packed<bf16, 8>(static_cast<bf16*>(base) + (row * a.D + d) * a.S + s + k, f);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kS; k += 4)
        store_states(base, row, a, d, s + k, live, is_bf16, make_float4(v[k / 2].x, v[k / 2].y, v[k / 2 + 1].x, v[k / 2 + 1].y));
}

// Sums kValues values over the lanes that differ in the bits from kBit up to kEnd.  While there are several values each
// step halves them: a lane keeps the upper half where its bit is set.  Returns the number of the first value that is
// left (of max(1, kValues / lanes)); where one is left before the lanes are done, the lanes beyond hold it too.
template <int kValues, int kBit, int kEnd>
__device__ __forceinline__ int spread_sum(float (&v)[kValues]) {
    if constexpr (kBit >= kEnd) {
        return 0;
    } else if constexpr (kValues == 1) {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], kBit);
        return spread_sum<1, 2 * kBit, kEnd>(v);
    } else {
        constexpr int kHalf = kValues / 2;
        const bool up = threadIdx.x & kBit;
        float w[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            const float mine = up ? v[i + kHalf] : v[i], other = up ? v[i] : v[i + kHalf];
            w[i] = mine + __shfl_xor_sync(0xffffffffu, other, kBit);
        }
        const int at = spread_sum<kHalf, 2 * kBit, kEnd>(w);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) v[i] = w[i];
        return (up ? kHalf : 0) + at;
    }
}

inline dim3 slot_grid(int tiles, int64_t slots) {
    const int64_t y = std::min<int64_t>(slots, 65535);
    return dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(y), static_cast<unsigned>((slots + y - 1) / y));
}
// ssm_fwd.cu, ssm_bwd.cu
int fwd_shift(int64_t T, int D, int S, int G, int time_block);
la_status run_fwd(Args a, int32_t dtype, cudaStream_t s);
la_status run_bwd(Args a, int32_t dtype, cudaStream_t s);
int bwd_width(int S);
int64_t bwd_blocks(int64_t T, int32_t N);
int bwd_parts(int64_t T, int32_t N, int D, int S, int G);

}  // namespace ssm
}  // namespace la
