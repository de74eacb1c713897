// sconv.cu -- the short causal convolution with an activation (sconv_fwd, sconv_bwd, sconv_decode).
//
// Per channel of each sequence, x_s for s < 0 being the initial state's rows:
//
//   p_t = b + sum_j w_j x_{t - (W - 1) + j},  y_t = act(p_t);
//   dp_t = dy_t act'(p_t),  dx_t = sum_j w_j dp_{t + (W - 1) - j} (+ the final state's gradient),
//   dw_j = sum_t dp_t x_{t - (W - 1) + j},  db = sum_t dp_t.
//
// The sums over the tokens apart, every token needs its W - 1 neighbours only.  A CTA takes blocks of 128
// tokens x 64 channels (with their W - 1 rows before, and after in the backward) into shared memory by TMA,
// the next block on its way while this one is worked on; each warp walks a span of 32 tokens (16 in the
// backward), each lane two channels with the window in registers.  A CTA keeps to one channel tile: the taps stay in registers, and in the
// backward (which recomputes p) so do the sums of dw and db over all its blocks, which a second kernel adds
// over the CTAs in order.  Rows that TMA cannot move go through the same shared memory with plain loads.
// The forward is bound by its bytes (2 rows): 8 x 8192 x 4096 bf16, W = 4, in 184 us, 5.8 TB/s (87 % of the measured
// copy rate).  The backward (3 rows, and 20 bytes a channel and CTA of partial sums) takes 128 us for a skewed batch
// of 49344 x 2048, 4.7 TB/s (71 %): its arithmetic (some 20 instructions an element, two of them special functions, a fifth
// of them repeated at the spans' ends) and the latency of each token's chain share the time with the bytes.
#include <algorithm>
#include <type_traits>

#include "mixer.cuh"

namespace {

using namespace la;
using namespace la::mixer;

constexpr int kDecodeThreads = 128;
constexpr int kBlock = 128;  // tokens of a block
// Warps of a CTA, one span of the block each.  Longer spans repeat less (W - 1 tokens of a span are looked at twice
// in the backward), more warps hide more: 8 x 8192 x 4096 bf16 forward 184 us with 4 warps, 209 with 8; the skewed
// batch of 49344 x 2048 backward 8 % less with 8 than with 4.
template <bool kBackward>
constexpr int warps() { return kBackward ? 8 : 4; }
constexpr int kChannels = 64;                          // of a CTA, two a lane
constexpr int kSms = 152;
constexpr uint64_t kWaitNs = 1000000000ull;

struct Args {
    const void *x, *w, *b, *cu, *s0, *dy, *dfin;
    int64_t x_st, y_st, dy_st, dx_st, T;
    int cu64, N, D, w_bf16, act;
    const int32_t* idx;
    int64_t pool;
    void *y, *fin, *dx, *ds0;
    float* part;     // [columns][W + 1][D]: dw_0 .. dw_{W-1}, db
    int32_t* status;
    int tiles, columns;  // channel tiles; CTAs of a tile
    int64_t slots;
    int tma, pair;   // inputs can move by TMA; results can be stored in pairs
};

// The state slot of sequence i, or false when its index is outside the pool.
__device__ __forceinline__ bool state_slot(const Args& a, int i, int64_t& slot) {
    slot = i;
    if (!a.idx) return true;
    slot = a.idx[i];
    if (slot >= 0 && slot < a.pool) return true;
    raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
    return false;
}

// Channels d, d + 1 of one row, below D.
template <typename T>
__device__ __forceinline__ float2 row2(const void* base, int64_t at, int d, int D) {
    const T* p = static_cast<const T*>(base) + at;
    return make_float2(d < D ? to_f(p[d]) : 0.f, d + 1 < D ? to_f(p[d + 1]) : 0.f);
}
template <typename T>
__device__ __forceinline__ void put_row2(void* base, int64_t at, int d, int D, float2 v) {
    T* p = static_cast<T*>(base) + at + d;
    if (d < D) p[0] = from_f<T>(v.x);
    if (d + 1 < D) p[1] = from_f<T>(v.y);
}
// Two channels, stored as a pair.
template <typename T>
__device__ __forceinline__ void put2(T* p, float2 v) {
    if (sizeof(T) == 4) *reinterpret_cast<float2*>(p) = v;
    else *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ float2 staged2(const T* p) {
    if (sizeof(T) == 4) return *reinterpret_cast<const float2*>(p);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The input at place pos of the sequence that starts at `first`: a token, or a row of the state before it.
template <typename X, int W>
__device__ __forceinline__ float2 input_at(const Args& a, int64_t first, int64_t slot, int64_t pos, int d) {
    if (pos >= 0) return row2<X>(a.x, (first + pos) * a.x_st, d, a.D);
    return a.s0 ? row2<X>(a.s0, (slot * (W - 1) + (W - 1) + pos) * a.D, d, a.D) : make_float2(0.f, 0.f);
}

template <int W>
__device__ __forceinline__ void load_taps(float2 (&w)[W], float2& bias, const Args& a, int d) {
    const bool in0 = d < a.D, in1 = d + 1 < a.D;
#pragma unroll
    for (int j = 0; j < W; ++j)
        w[j] = make_float2(in0 ? load_any(a.w, static_cast<int64_t>(d) * W + j, a.w_bf16) : 0.f,
                           in1 ? load_any(a.w, static_cast<int64_t>(d + 1) * W + j, a.w_bf16) : 0.f);
    bias = a.b ? make_float2(in0 ? load_any(a.b, d, a.w_bf16) : 0.f, in1 ? load_any(a.b, d + 1, a.w_bf16) : 0.f) : make_float2(0.f, 0.f);
}

struct Maps {
    CUtensorMap x, dy;
};

// Rows staged for a block: the W - 1 before it, its own, and in the backward the W - 1 after it.
template <int W, bool kBackward>
constexpr int x_rows() { return kBlock + (W - 1) * (kBackward ? 2 : 1); }
template <int W, bool kBackward>
constexpr int dy_rows() { return kBackward ? kBlock + W - 1 : 0; }
template <typename X, int W, bool kBackward>
constexpr size_t stage_bytes() { return (x_rows<W, kBackward>() + dy_rows<W, kBackward>()) * kChannels * sizeof(X); }
// 16-bit operands leave room for two stages and enough CTAs; 32-bit ones take more CTAs of one.
template <typename X>
constexpr int stages() { return sizeof(X) == 2 ? 2 : 1; }

struct Shared {
    uint64_t bar[2];
    SeqBlock block[2];
};

// The blocks of one CTA, one after the other, in shared memory.
template <typename X, int W, bool kBackward>
struct Blocks {
    const Args& a;
    const Maps& maps;
    X* stage;
    Shared& sh;
    int tile;

    __device__ __forceinline__ X* x_at(int st) const { return stage + st * (stage_bytes<X, W, kBackward>() / sizeof(X)); }
    __device__ __forceinline__ X* dy_at(int st) const { return x_at(st) + x_rows<W, kBackward>() * kChannels; }

    // By warp 0: finds the block of a slot and starts its rows on their way.
    __device__ __forceinline__ void fetch(int64_t slot, int st) const {
        const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, slot);
        if ((threadIdx.x & 31) == 0) {
            sh.block[st] = b;
            if (a.tma) {
                const bool any = b.seq >= 0 && b.count > 0;
                mbar_arrive_expect_tx(&sh.bar[st], any ? static_cast<uint32_t>(stage_bytes<X, W, kBackward>()) : 0u);
                if (any) {
                    tile_load(x_at(st), &maps.x, &sh.bar[st], tile * kChannels, b.start - (W - 1));
                    if (kBackward) tile_load(dy_at(st), &maps.dy, &sh.bar[st], tile * kChannels, b.start);
                }
            }
        }
        __syncwarp();
    }
    // Without TMA, by the whole CTA: rows outside the batch are not read.
    __device__ __forceinline__ void copy(int st) const {
        const SeqBlock& b = sh.block[st];
        if (b.seq < 0 || b.count == 0) return;
        copy_rows(x_at(st), a.x, a.x_st, b.start - (W - 1), x_rows<W, kBackward>());
        if (kBackward) copy_rows(dy_at(st), a.dy, a.dy_st, b.start, dy_rows<W, kBackward>());
    }
    __device__ __forceinline__ void copy_rows(X* to, const void* base, int64_t stride, int first, int rows) const {
#pragma unroll 4
        for (int e = threadIdx.x; e < rows * kChannels; e += 32 * warps<kBackward>()) {
            const int r = e / kChannels, c = e % kChannels, d = tile * kChannels + c;
            const int64_t t = static_cast<int64_t>(first) + r;
            if (t >= 0 && t < a.T && d < a.D) to[e] = static_cast<const X*>(base)[t * stride + d];
        }
    }
    // Calls f(block, x rows, dy rows) for every slot of this CTA.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        const int warp = threadIdx.x >> 5;
        const int64_t first = blockIdx.x / a.tiles;
        if (threadIdx.x == 0) {
            mbar_init(&sh.bar[0], 1);
            mbar_init(&sh.bar[1], 1);
        }
        fence_mbar_init();
        __syncthreads();
        const int depth = a.tma ? stages<X>() : 1;
        if (warp == 0)
            for (int k = 0; k < depth; ++k)
                if (first + static_cast<int64_t>(k) * a.columns < a.slots) fetch(first + static_cast<int64_t>(k) * a.columns, k);
        uint32_t parity = 0;
        int st = 0;
        for (int64_t slot = first; slot < a.slots; slot += a.columns) {
            if (a.tma) {
                if (!mbar_wait(&sh.bar[st], parity, kWaitNs)) raise_status(a.status, LA_ERR_TIMEOUT);
            } else {
                __syncthreads();
                copy(st);
                __syncthreads();
            }
            f(sh.block[st], x_at(st), dy_at(st));
            __syncthreads();  // everybody is done with this stage
            const int64_t ahead = slot + static_cast<int64_t>(depth) * a.columns;
            if (warp == 0 && ahead < a.slots) fetch(ahead, st);
            if (++st == depth) {
                st = 0;
                parity ^= 1;
            }
        }
    }
};

template <typename X, int W, int kAct>
__global__ void __launch_bounds__(32 * warps<false>()) sconv_fwd_kernel(const Args a, const __grid_constant__ Maps maps) {
    constexpr int kWarps = warps<false>(), kThreads = 32 * kWarps, kSpan = kBlock / kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int tile = blockIdx.x % a.tiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = tile * kChannels + 2 * lane;
    if (tile == 0)
        for (int64_t i = (blockIdx.x / a.tiles) * static_cast<int64_t>(kThreads) + threadIdx.x; i < a.N; i += static_cast<int64_t>(a.columns) * kThreads)
            check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
    float2 w[W], bias;
    load_taps<W>(w, bias, a, d);
    Blocks<X, W, false> blocks{a, maps, reinterpret_cast<X*>(smem), sh, tile};
    blocks.each([&](const SeqBlock& b, const X* xs, const X*) {
        int64_t slot;
        if (b.seq < 0 || !state_slot(a, b.seq, slot)) return;
        const int k0 = warp * kSpan, n = min(kSpan, b.count - k0);
        if (n > 0) {
            float2 win[W];
            const X* px = xs + k0 * kChannels + 2 * lane;  // row 0: the token W - 1 before the span
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                win[j + 1] = b.c == 0 && warp == 0 ? input_at<X, W>(a, b.first, slot, j - (W - 1), d) : staged2(px + j * kChannels);
            px += (W - 1) * kChannels;
            X* py = static_cast<X*>(a.y) + (static_cast<int64_t>(b.start) + k0) * a.y_st;
            const bool in = d < a.D;
            auto token = [&](int k, auto pair) {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1];
                win[W - 1] = staged2(px + k * kChannels);
                float2 p = bias;
#pragma unroll
                for (int j = 0; j < W; ++j) p = fma2(w[j], win[j], p);
                const float2 y = act_fwd2<kAct>(p);
                if (!pair) put_row2<X>(py, 0, d, a.D, y);
                else if (in) put2<X>(py + d, y);
                py += a.y_st;
            };
            if (n == kSpan && a.pair) {
#pragma unroll 2
                for (int k = 0; k < kSpan; ++k) token(k, std::true_type());
            } else {
                for (int k = 0; k < n; ++k) token(k, std::false_type());
            }
        }
        // The sequence's last W - 1 inputs.  With a pool they replace the rows that the sequence started from,
        // which only this thread reads: they reach the first W - 1 tokens, and kSpan is no less.
        if (b.c == 0 && warp == 0 && (a.fin || a.idx)) {
            float2 f[W - 1];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) f[j] = input_at<X, W>(a, b.first, slot, static_cast<int64_t>(b.len) - (W - 1) + j, d);
            void* to = a.idx ? const_cast<void*>(a.s0) : a.fin;
            const int64_t row = (a.idx ? slot : b.seq) * (W - 1);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) put_row2<X>(to, (row + j) * a.D, d, a.D, f[j]);
        }
    });
}

template <typename X, int W, int kAct>
__global__ void __launch_bounds__(32 * warps<true>()) sconv_bwd_kernel(const Args a, const __grid_constant__ Maps maps) {
    constexpr int kWarps = warps<true>(), kThreads = 32 * kWarps, kSpan = kBlock / kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int tile = blockIdx.x % a.tiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = tile * kChannels + 2 * lane;
    if (tile == 0)
        for (int64_t i = (blockIdx.x / a.tiles) * static_cast<int64_t>(kThreads) + threadIdx.x; i < a.N; i += static_cast<int64_t>(a.columns) * kThreads)
            check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
    float2 w[W], bias, dw[W], db = make_float2(0.f, 0.f);
    load_taps<W>(w, bias, a, d);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = make_float2(0.f, 0.f);
    Blocks<X, W, true> blocks{a, maps, reinterpret_cast<X*>(smem), sh, tile};
    blocks.each([&](const SeqBlock& b, const X* xs, const X* dys) {
        if (b.seq < 0) return;
        const int k0 = warp * kSpan, n = min(kSpan, b.count - k0);
        // the gradient that the final state's rows bring to the place f - (W - 1) before the sequence's end
        auto add_final = [&](float2 v, int64_t f) {
            if (a.dfin && f >= 0) {
                const float2 e = row2<X>(a.dfin, (b.seq * static_cast<int64_t>(W - 1) + f) * a.D, d, a.D);
                v.x += e.x;
                v.y += e.y;
            }
            return v;
        };
        float2 dp0[W - 1];  // dp of the span's first tokens: what the state's rows reach
        if (n > 0) {
            const int64_t p0 = static_cast<int64_t>(b.c) * kBlock + k0;
            X* pdx = static_cast<X*>(a.dx) + (static_cast<int64_t>(b.start) + k0) * a.dx_st;
            const int left = static_cast<int>(min(b.len - p0, static_cast<int64_t>(kSpan + W - 1)));  // tokens to the sequence's end
            float2 win[W], dp[W];
            const X* px = xs + k0 * kChannels + 2 * lane;
            const X* pd = dys + k0 * kChannels + 2 * lane;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                win[j + 1] = b.c == 0 && warp == 0 ? input_at<X, W>(a, b.first, b.seq, j - (W - 1), d) : staged2(px + j * kChannels);
                dp[j + 1] = make_float2(0.f, 0.f);
            }
            px += (W - 1) * kChannels;
            // `whole`: every token that the span reads is in the sequence, so that nothing is masked, and results are
            // stored in pairs
            const bool in = d < a.D;
            auto walk = [&](auto whole) {
                // one token further: win ends with token k, dp with its dp (0 beyond the end)
                auto step = [&](int k) {
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) {
                        win[j] = win[j + 1];
                        dp[j] = dp[j + 1];
                    }
                    win[W - 1] = staged2(px + k * kChannels);
                    const float2 dy = staged2(pd + k * kChannels);
                    float2 p = bias, s;
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fma2(w[j], win[j], p);
                    act_grad2<kAct>(p, s);
                    dp[W - 1] = mul2(dy, s);
                    if (!whole && k >= left) dp[W - 1] = win[W - 1] = make_float2(0.f, 0.f);
                };
                auto emit = [&](int k) {  // dx of token k, W - 1 behind
                    if (!whole && k >= n) return;
                    float2 dx = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < W; ++j) dx = fma2(w[j], dp[W - 1 - j], dx);
                    if (!whole) put_row2<X>(pdx, 0, d, a.D, add_final(dx, p0 + k - (static_cast<int64_t>(b.len) - (W - 1))));
                    else if (in) put2<X>(pdx + d, dx);
                    pdx += a.dx_st;
                };
                auto sum = [&]() {
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j] = fma2(dp[W - 1], win[j], dw[j]);
                    db = add2(db, dp[W - 1]);
                };
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                    step(k);
                    sum();
                    dp0[k] = dp[W - 1];
                }
#pragma unroll 8
                for (int k = W - 1; k < kSpan; ++k) {
                    step(k);
                    sum();
                    emit(k - (W - 1));
                }
#pragma unroll
                for (int k = kSpan; k < kSpan + W - 1; ++k) {
                    step(k);
                    emit(k - (W - 1));
                }
            };
            if (left >= kSpan + W - 1 && a.pair) walk(std::true_type());
            else walk(std::false_type());
        } else {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) dp0[k] = make_float2(0.f, 0.f);
        }
        // d(initial state): the row at place s - (W - 1) is tap s - t of token t <= s
        if (b.c == 0 && a.ds0 && warp == 0) {
#pragma unroll
            for (int s = 0; s < W - 1; ++s) {
                float2 ds = make_float2(0.f, 0.f);
#pragma unroll
                for (int t = 0; t <= s; ++t) ds = fma2(w[s - t], dp0[t], ds);
                ds = add_final(ds, static_cast<int64_t>(s) - b.len);
                put_row2<X>(a.ds0, (b.seq * static_cast<int64_t>(W - 1) + s) * a.D, d, a.D, ds);
            }
        }
    });
    float2(*red)[W + 1][32] = reinterpret_cast<float2(*)[W + 1][32]>(smem);  // the stages are free
    static_assert(sizeof(float2) * kWarps * (W + 1) * 32 <= stage_bytes<X, W, true>(), "the sums fit a stage");
#pragma unroll
    for (int j = 0; j < W; ++j) red[warp][j][lane] = dw[j];
    red[warp][W][lane] = db;
    __syncthreads();
    for (int e = threadIdx.x; e < (W + 1) * kChannels; e += kThreads) {
        const int j = e / kChannels, c = e % kChannels;
        if (tile * kChannels + c >= a.D) continue;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += reinterpret_cast<const float*>(red[i][j])[c];
        a.part[(static_cast<int64_t>(blockIdx.x / a.tiles) * (W + 1) + j) * a.D + tile * kChannels + c] = s;
    }
}

// dw[d][j] and db[d]: the partial sums of all columns.  A CTA takes 32 channels of one j; its 32 warps
// take every 32nd column, in order.
template <int W>
__global__ void __launch_bounds__(1024) sconv_sum_kernel(const float* part, int64_t columns, int D, void* dw, void* db,
                                                         int w_bf16) {
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.y;
    const int d = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (d < D) s = strided_sum<2>(part + static_cast<int64_t>(j) * D + d, static_cast<int64_t>(W + 1) * D, warp, columns, 32);
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sh[i][lane];
        if (j < W) store_any(dw, static_cast<int64_t>(d) * W + j, w_bf16, s);
        else if (db) store_any(db, d, w_bf16, s);
    }
}

// One token: 512 x 8192 bf16 in 9.5 us from L2, 13 from memory, bound by its bytes (2 W rows) once the taps of a
// thread's channels come in wide loads (19 us one by one).
template <typename T, int kVec, int W>
__device__ __forceinline__ void load_run(float (&w)[kVec * W], const void* base, int d) {
#pragma unroll
    for (int r = 0; r < W; ++r) {
        Packed<T, kVec> q;
        q.load(static_cast<const T*>(base) + static_cast<int64_t>(d) * W + r * kVec);
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[r * kVec + i] = q.get(i);
    }
}

template <typename X, int W, int kVec>
__global__ void __launch_bounds__(kDecodeThreads) sconv_decode_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = (blockIdx.x * kDecodeThreads + threadIdx.x) * kVec;
    int64_t slot;
    if (i >= a.N || d >= a.D || !state_slot(a, i, slot)) return;
    X* st = static_cast<X*>(const_cast<void*>(a.s0)) + slot * (W - 1) * a.D + d;
    Packed<X, kVec> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j].load(st + static_cast<int64_t>(j) * a.D);
    in[W - 1].load(static_cast<const X*>(a.x) + i * a.x_st + d);
    float w[kVec * W], y[kVec];  // the taps of the thread's channels follow one another
    if (a.w_bf16) load_run<bf16, kVec, W>(w, a.w, d);
    else load_run<float, kVec, W>(w, a.w, d);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        float p = a.b ? load_any(a.b, d + e, a.w_bf16) : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(w[e * W + j], in[j].get(e), p);
        y[e] = act_fwd(a.act, p);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float v[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = in[j + 1].get(e);
        store_packed<X, kVec>(st + static_cast<int64_t>(j) * a.D, v);
    }
    store_packed<X, kVec>(static_cast<X*>(a.y) + i * a.y_st + d, y);
}

// CTAs of a channel tile: what the GPU holds at once (by shared memory, 3 or 6 an SM), no more than slots.
int64_t bwd_columns(int64_t T, int32_t N, int32_t D) {
    const int64_t tiles = (D + kChannels - 1) / kChannels;
    return std::max<int64_t>(1, std::min<int64_t>(T / kBlock + N, kSms * 3 / tiles));
}

template <auto kKernel>
la_status launch_blocks(int threads, size_t smem, const Args& a, const Maps& maps, cudaStream_t s) {
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    kKernel<<<static_cast<unsigned>(a.tiles * a.columns), threads, smem, s>>>(a, maps);
    return launched();
}

template <typename X, int W>
la_status run_blocks(Args& a, bool bwd, int32_t xd, cudaStream_t s) {
    a.tiles = (a.D + kChannels - 1) / kChannels;
    a.slots = a.T / kBlock + a.N;
    if (a.slots == 0) return LA_OK;
    a.columns = static_cast<int>(bwd ? bwd_columns(a.T, a.N, a.D)
                                     : std::max<int64_t>(1, std::min<int64_t>(a.slots, kSms * 6 / a.tiles)));
    Maps maps = {};
    a.tma = tileable(a.x, a.x_st, a.T, a.D, xd) && (!bwd || tileable(a.dy, a.dy_st, a.T, a.D, xd));
    if (a.tma && bwd)
        a.tma = tile_map(&maps.x, a.x, a.x_st, a.T, a.D, xd, kChannels, x_rows<W, true>()) &&
                tile_map(&maps.dy, a.dy, a.dy_st, a.T, a.D, xd, kChannels, dy_rows<W, true>());
    else if (a.tma)
        a.tma = tile_map(&maps.x, a.x, a.x_st, a.T, a.D, xd, kChannels, x_rows<W, false>());
    const void* out = bwd ? a.dx : a.y;
    const int64_t stride = bwd ? a.dx_st : a.y_st;
    a.pair = a.D % 2 == 0 && aligned_to(out, 2 * sizeof(X)) && (a.T == 1 || stride % 2 == 0);
    const int depth = a.tma ? stages<X>() : 1;
    auto start = [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        return bwd ? launch_blocks<sconv_bwd_kernel<X, W, kAct>>(32 * warps<true>(), depth * stage_bytes<X, W, true>(), a, maps, s)
                   : launch_blocks<sconv_fwd_kernel<X, W, kAct>>(32 * warps<false>(), depth * stage_bytes<X, W, false>(), a, maps, s);
    };
    if (a.act == LA_ACT_SILU) return start(std::integral_constant<int, LA_ACT_SILU>());
    if (a.act == LA_ACT_SIGMOID) return start(std::integral_constant<int, LA_ACT_SIGMOID>());
    return start(std::integral_constant<int, LA_ACT_NONE>());
}

// Four channels a lane where every operand's rows start on four of its elements.
template <typename X, int W>
la_status run_decode(const Args& a, cudaStream_t s) {
    if (a.N == 0) return LA_OK;
    const int bytes = 4 * static_cast<int>(sizeof(X));
    auto ok = [&](const void* p, int64_t st) { return aligned_to(p, bytes) && st % 4 == 0; };
    const bool four = a.D % 4 == 0 && ok(a.x, a.x_st) && ok(a.y, a.y_st) && ok(a.s0, 0) && aligned_to(a.w, a.w_bf16 ? 8 : 16);
    const int ny = std::min(a.N, 65535), nz = (a.N + ny - 1) / ny, width = kDecodeThreads * (four ? 4 : 1);
    const dim3 grid((a.D + width - 1) / width, ny, nz);
    if (four) sconv_decode_kernel<X, W, 4><<<grid, kDecodeThreads, 0, s>>>(a);
    else sconv_decode_kernel<X, W, 1><<<grid, kDecodeThreads, 0, s>>>(a);
    return launched();
}

enum Which { kFwd, kBwd, kDecode };

template <typename X, int W>
la_status run(Args& a, Which w, int32_t xd, cudaStream_t s) {
    return w == kDecode ? run_decode<X, W>(a, s) : run_blocks<X, W>(a, w == kBwd, xd, s);
}

la_status dispatch(Args& a, int W, int32_t xd, Which w, cudaStream_t s) {
    if (xd == LA_DTYPE_BF16) return W == 2 ? run<bf16, 2>(a, w, xd, s) : W == 3 ? run<bf16, 3>(a, w, xd, s) : run<bf16, 4>(a, w, xd, s);
    return W == 2 ? run<float, 2>(a, w, xd, s) : W == 3 ? run<float, 3>(a, w, xd, s) : run<float, 4>(a, w, xd, s);
}

la_status check(int32_t D, int32_t W, int32_t xd, int32_t wd, int32_t act, const void* w, const void* b) {
    if (D <= 0) return LA_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || !known_dtype(xd) || !known_dtype(wd)) return LA_ERR_UNSUPPORTED;
    if (act < LA_ACT_NONE || act > LA_ACT_SIGMOID) return LA_ERR_INVALID_ARG;
    if (!w || !aligned_to(w, dtype_size(wd)) || !good_optional(b, wd)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

}  // namespace

extern "C" {

size_t la_sconv_bwd_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t W) {
    if (T < 0 || N < 0 || D <= 0 || W < 2 || W > 4) return 0;
    return (static_cast<size_t>(bwd_columns(T, N, D)) * (W + 1) * D * 4 + 255) & ~size_t(255);
}

la_status sconv_fwd(const la_sconv_fwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if ((st = check(p->D, p->W, p->x_dtype, p->weight_dtype, p->activation, p->weight, p->bias)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->y, p->y_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_optional(p->initial_state, p->x_dtype) || !good_optional(p->final_state, p->x_dtype))
        return LA_ERR_INVALID_ARG;
    if (p->state_indices && (!aligned_to(p->state_indices, 4) || !p->initial_state || p->final_state || p->state_pool_size <= 0))
        return LA_ERR_INVALID_ARG;
    if (rows_meet(p->x, p->x_stride_t, p->y, p->y_stride_t, p->T, p->D, p->x_dtype)) return LA_ERR_INVALID_ARG;  // neighbours read x
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D; a.act = p->activation;
    a.s0 = p->initial_state; a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.y = p->y; a.y_st = p->y_stride_t; a.fin = p->final_state; a.status = p->status;
    return dispatch(a, p->W, p->x_dtype, kFwd, static_cast<cudaStream_t>(stream));
}

la_status sconv_bwd(const la_sconv_bwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if ((st = check(p->D, p->W, p->x_dtype, p->weight_dtype, p->activation, p->weight, p->bias)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->dy, p->dy_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->dx, p->dx_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_optional(p->initial_state, p->x_dtype) || !good_optional(p->d_final_state, p->x_dtype) ||
        !good_optional(p->d_initial_state, p->x_dtype))
        return LA_ERR_INVALID_ARG;
    if (!p->d_weight || !aligned_to(p->d_weight, dtype_size(p->weight_dtype)) || (p->bias && !p->d_bias) ||
        !good_optional(p->d_bias, p->weight_dtype))
        return LA_ERR_INVALID_ARG;
    if ((st = check_workspace(p->workspace, p->workspace_bytes, la_sconv_bwd_workspace_bytes(p->T, p->N, p->D, p->W))) != LA_OK)
        return st;
    if (rows_meet(p->x, p->x_stride_t, p->dx, p->dx_stride_t, p->T, p->D, p->x_dtype) ||
        rows_meet(p->dy, p->dy_stride_t, p->dx, p->dx_stride_t, p->T, p->D, p->x_dtype))
        return LA_ERR_INVALID_ARG;  // neighbours read x and dy
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D; a.act = p->activation;
    a.s0 = p->initial_state; a.dy = p->dy; a.dy_st = p->dy_stride_t; a.dfin = p->d_final_state;
    a.dx = p->dx; a.dx_st = p->dx_stride_t; a.ds0 = p->d_initial_state;
    a.part = static_cast<float*>(p->workspace); a.status = p->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = dispatch(a, p->W, p->x_dtype, kBwd, s)) != LA_OK) return st;
    const dim3 grid((a.D + 31) / 32, p->W + (p->bias ? 1 : 0));
    const int64_t columns = a.slots ? a.columns : 0;
    void* db = p->bias ? p->d_bias : nullptr;
    if (p->W == 2) sconv_sum_kernel<2><<<grid, 1024, 0, s>>>(a.part, columns, a.D, p->d_weight, db, a.w_bf16);
    else if (p->W == 3) sconv_sum_kernel<3><<<grid, 1024, 0, s>>>(a.part, columns, a.D, p->d_weight, db, a.w_bf16);
    else sconv_sum_kernel<4><<<grid, 1024, 0, s>>>(a.part, columns, a.D, p->d_weight, db, a.w_bf16);
    return launched();
}

la_status sconv_decode(const la_sconv_decode_params* p, void* stream) {
    if (!p || p->N < 0) return LA_ERR_INVALID_ARG;
    la_status st = check(p->D, p->W, p->x_dtype, p->weight_dtype, p->activation, p->weight, p->bias);
    if (st != LA_OK) return st;
    if (!p->state_pool || !good_optional(p->state_pool, p->x_dtype) || p->state_pool_size <= 0) return LA_ERR_INVALID_ARG;
    if (p->state_indices ? !aligned_to(p->state_indices, 4) : p->state_pool_size < p->N) return LA_ERR_INVALID_ARG;
    if (!good_rows(p->x, p->x_stride_n, p->N, p->D, p->x_dtype, false) ||
        !good_rows(p->y, p->y_stride_n, p->N, p->D, p->x_dtype, true))
        return LA_ERR_INVALID_ARG;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_n; a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.N = p->N; a.D = p->D; a.act = p->activation;
    a.s0 = p->state_pool; a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.y = p->y; a.y_st = p->y_stride_n; a.status = p->status;
    return dispatch(a, p->W, p->x_dtype, kDecode, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
