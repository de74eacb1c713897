// ssm_bwd.cu -- the selective scan's backward (ssm.cuh has the formulas).
//
// Time is cut into blocks of 64 tokens from each sequence's start.  A first launch leaves what each block makes of a zero
// gradient behind it, and its steps' sum; a second one goes along each sequence from its end, which gives the gradient
// behind every block; then all blocks are worked on side by side.  Blocks are fixed by the sequence alone, so the gradients
// of its inputs do not depend on the batch around it.
//
// Within a block 16 tokens are taken at a time from the end, the state before them being the forward's checkpoint.  A warp
// goes forward once, leaving the states before every fourth token in shared memory (and p, for dz), then takes four tokens
// at a time from the end: forward again with states and decays kept in registers, then back.  dB and dC are summed over a
// thread's channels, the warp's, the CTA's, and by a later launch over the CTAs that share a group; dA, d skip and d bias over
// a block's tokens, a CTA's blocks and then the CTAs, all in an order that the shape fixes.  What the CTAs leave of dB and dC is
// 8 S bytes a token for each tile of 128, 64 or 32 channels (S up to 16, 32 and 64), written and read once: 1 byte a channel and
// token for 16 states, 4 for 32, 16 for 64, where x has 2 in bf16 and the checkpoints S / 4.
#include "ssm.cuh"

namespace la {
namespace ssm {
namespace {

constexpr int kShift = 6, kBlock = 1 << kShift;
static_assert(kBlock % kSave == 0, "a block's parts are what the forward saved states for");

// ---------------------------------------------------------------- the gradient behind each block
// As in the forward, a lane has one channel with kS of its states.
constexpr int kTok = 32;

template <typename X, int kS, int Q>
struct Stage {
    static constexpr int kW = 32 / Q, kSP = kS * Q;
    X rows[2][3][kTok * kW];  // dt, dy, z
    X states[2][kTok * kSP];  // C
    float wide[sizeof(X) == 4 ? 4 : kTok * kSP];
};

template <typename X, int kS, int Q, bool kGate>
__global__ void __launch_bounds__(32) ssm_block_gradient_kernel(const Args a) {
    typedef Stage<X, kS, Q> Sm;
    constexpr int kW = Sm::kW, kSP = Sm::kSP, kPairs = kS / 2;
    __shared__ __align__(16) Sm sm;
    const int lane = threadIdx.x, q = lane / kW, ch = lane % kW;
    const int64_t slot = this_slot();
    if (slot >= slots_for(a.T, a.N, kShift)) return;
    const SeqBlock blk = find_slot(a, kShift, slot);
    if (blk.seq < 0 || blk.count == 0) return;
    const Tile tile = tile_of(a, blockIdx.x, kW);
    const int d = tile.ch + ch, s0 = kS * q;
    const bool live = ch < tile.n;

    typedef Rows<X, kW, 32, kTok> RowsOf;
    const RowsOf dt_rows(a.dt, blk.start * a.dt_st + tile.ch, a.dt_st, tile.n, a.vec), dy_rows(a.dy, blk.start * a.dy_st + tile.ch, a.dy_st, tile.n, a.vec),
        z_rows(a.z, blk.start * a.z_st + tile.ch, a.z_st, tile.n, a.vec);
    const Rows<X, kSP, 32, kTok> c_rows(a.c, blk.start * a.c_st + tile.group * a.c_sg, a.c_st, a.S, a.vec);
    auto load = [&](int buf, int t) {
        if (t >= 0) {
            const int rows = blk.count - t;
            dt_rows.stage(sm.rows[buf][0], t, rows);
            dy_rows.stage(sm.rows[buf][1], t, rows);
            if (kGate) z_rows.stage(sm.rows[buf][2], t, rows);
            c_rows.stage(sm.states[buf], t, rows);
        }
        cp_async_commit();
    };
    int t0 = (blk.count - 1) / kTok * kTok, buf = 0;
    load(0, t0);
    float2 A2[kPairs], g[kPairs];
    load_lane_states<kS>(A2, a.A, 0, a, d, s0, live, 0);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        A2[k] = mul2(A2[k], both(kLog2e));
        g[k] = both(0.f);
    }
    const float bias = live && a.bias ? a.bias[d] : 0.f;
    float sum = 0.f;
    for (; t0 >= 0; t0 -= kTok, buf ^= 1) {
        load(buf ^ 1, t0 - kTok);
        cp_async_wait<1>();
        __syncwarp();
        const int n = min(kTok, blk.count - t0);
        const float* cs;
        if constexpr (sizeof(X) == 4) {
            cs = sm.states[buf];
        } else {
#pragma unroll
            for (int j = 0; j < kTok * kSP / 128; ++j) {
                const int i = 4 * (lane + 32 * j);
                *reinterpret_cast<float4*>(sm.wide + i) = load4<X>(sm.states[buf], i, 4, 1);
            }
            __syncwarp();
            cs = sm.wide;
        }
        cs += s0;
        const X *ds = sm.rows[buf][0] + ch, *ys = sm.rows[buf][1] + ch, *zs = sm.rows[buf][2] + ch;
        struct Pair {  // two tokens' steps and gradients of p
            float2 dt, dp;
        };
        auto prepare = [&](int r) {
            Pair t;
            const float2 raw = add2(make_float2(to_f(ds[r * kW]), to_f(ds[r * kW + kW])), both(bias)), sp = softplus2(raw);
            t.dt = make_float2(a.softplus ? sp.x : raw.x, a.softplus ? sp.y : raw.y);
            t.dp = make_float2(to_f(ys[r * kW]), to_f(ys[r * kW + kW]));
            if (kGate) t.dp = mul2(t.dp, act_fwd2<LA_ACT_SILU>(make_float2(to_f(zs[r * kW]), to_f(zs[r * kW + kW]))));
            return t;
        };
        auto token = [&](float dt, float dp, int r) {
            const float2 d2 = both(dt), p2 = both(dp);
#pragma unroll
            for (int k = 0; k < kPairs; k += 2) {
                const float4 c = *reinterpret_cast<const float4*>(cs + r * kSP + 2 * k);
                const float2 l0 = fma2(d2, A2[k], both(kEx2Low)), l1 = fma2(d2, A2[k + 1], both(kEx2Low));
                g[k] = mul2(make_float2(ex2(l0.x), ex2(l0.y)), fma2(p2, lo(c), g[k]));
                g[k + 1] = mul2(make_float2(ex2(l1.x), ex2(l1.y)), fma2(p2, hi(c), g[k + 1]));
            }
            sum += dt;
        };
        int r = n & ~1;
        if (n & 1) {
            const Pair t = prepare(n - 1 & ~1);  // the first of its two tokens
            token(t.dt.x, t.dp.x, n - 1);
        }
        Pair now = prepare(max(r - 2, 0));
#pragma unroll 2
        for (r -= 2; r >= 0; r -= 2) {
            const Pair next = prepare(max(r - 2, 0));
            token(now.dt.y, now.dp.y, r + 1);
            token(now.dt.x, now.dp.x, r);
            now = next;
        }
        __syncwarp();
    }
    store_lane_states<kS>(g, a.table, slot, a, d, s0, live, 0);
    if (live && q == 0) a.sums[slot * a.D + d] = sum;
}

__global__ void __launch_bounds__(128) ssm_join_back_kernel(const Args a) {
    const int64_t e = blockIdx.x * 128ll + threadIdx.x, DS = static_cast<int64_t>(a.D) * a.S;
    const int64_t i = this_slot();
    if (i >= a.N || e >= DS) return;
    const int64_t t0 = cu_load(a.cu, a.cu64, i), t1 = cu_load(a.cu, a.cu64, i + 1);
    if (blockIdx.x == 0 && threadIdx.x == 0) check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
    if (t0 < 0 || t1 < t0 || t1 > a.T) return;
    const int64_t blocks = (t1 - t0 + kBlock - 1) >> kShift, slot = (t0 >> kShift) + i;
    float g = a.dfin ? a.dfin[i * DS + e] : 0.f;
    const float A2 = a.A[e] * kLog2e;
    const int64_t d = e / a.S;
    constexpr int kAhead = 16;
    for (int64_t c = blocks - 1; c >= 0; c -= kAhead) {
        float loc[kAhead], sum[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            loc[k] = c >= k ? a.table[(slot + c - k) * DS + e] : 0.f;
            sum[k] = c >= k ? a.sums[(slot + c - k) * a.D + d] : 0.f;
        }
        g = walk_blocks(g, A2, sum, loc, [&](int k, float entering) {
            if (c >= k) a.table[(slot + c - k) * DS + e] = entering;
            return c >= k;
        });
    }
    if (a.ds0) a.ds0[i * DS + e] = g;
}

// ---------------------------------------------------------------- all gradients of a block
// A lane has four channels with four states each, Q lanes share the channels: what is summed over channels and what is
// summed over states then both have few lanes to cross.  65536 x 2048 x 16, gated, in 2.46 ms: 375 instructions a token of a warp
// (32 channels), 157 of them pairs of operations, with two warps a scheduler.
constexpr int kWarps = 4, kThreads = 32 * kWarps, kSub = kSave;

template <typename X, int Q>
struct Work {
    static constexpr int kW = 128 / Q, kTile = kWarps * kW, kSP = 4 * Q;  // channels of a warp, of a CTA; states
    static constexpr int kBufs = sizeof(X) == 4 ? 1 : 2;
    X rows[kBufs][4][kSub * kTile];   // x, dt, dy, z
    X states[kBufs][2][kSub * kSP];   // B, C
    float dt[kSub][kTile], u[kSub][kTile], dp[kSub][kTile], r[kSub][kTile];  // u: dt x, then du; r: p, then the sum of w A log2(e)
    float b[kSub][kSP], c[kSub][kSP];
    float4 h[kWarps][kSub / 4][4][32];  // the states before every fourth token
    float dbc[kWarps][kSub][2 * kSP];   // dB, dC of a warp's channels
    float4 ch[2][kThreads];             // d skip, d bias of the blocks so far, each thread's own
};

// Four consecutive floats of global memory that no other thread adds to.
__device__ __forceinline__ void add_to(float* p, float4 f, int vec, int n) {
    if (vec) {
        asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(f.x), "f"(f.y), "f"(f.z), "f"(f.w) : "memory");
        return;
    }
    const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p + i), "f"(v[i]) : "memory");
}
// store_thread_states's counterpart.
__device__ __forceinline__ void add_thread_states(const float2 (&v)[2][4], float* base, int64_t row, const Args& a, int d, int end, int s) {
    if (s >= a.S) return;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float* const at = base + (row * a.D + d + 2 * p) * a.S + s;
        if (d + 2 * p < end) add_to(at, make_float4(v[p][0].x, v[p][1].x, v[p][2].x, v[p][3].x), a.svec, a.S - s);
        if (d + 2 * p + 1 < end) add_to(at + a.S, make_float4(v[p][0].y, v[p][1].y, v[p][2].y, v[p][3].y), a.svec, a.S - s);
    }
}
__device__ __forceinline__ void add4(float4& to, const float2 (&v)[2]) {
    to = make_float4(to.x + v[0].x, to.y + v[0].y, to.z + v[1].x, to.w + v[1].y);
}

template <typename X, int Q, bool kGate>
__global__ void __launch_bounds__(kThreads, 2) ssm_block_kernel(const Args a) {
    typedef Work<X, Q> Wk;
    constexpr int kW = Wk::kW, kTile = Wk::kTile, kSP = Wk::kSP, kBufs = Wk::kBufs;
    extern __shared__ __align__(16) uint8_t raw_smem[];
    Wk& sm = *reinterpret_cast<Wk*>(raw_smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, q = lane % Q, cg = lane / Q;
    const int tiles = a.tiles_pg * a.G, part = blockIdx.x / tiles, tl = blockIdx.x - part * tiles;
    const Tile tile = tile_of(a, tl, kTile);
    const int cl = w * kW + 4 * cg;  // the thread's first channel within the tile
    const int d0 = tile.ch + cl, end = tile.ch + tile.n, s0 = 4 * q;
    // the four channels that this thread prepares and finishes, of every kRows-th row
    constexpr int kVecs = kTile / 4, kRows = kThreads / kVecs;
    const int c4 = tid % kVecs * 4, r4 = tid / kVecs, cn = tile.n - c4;
    float2 bias[2], skip[2], d_skip[2], d_bias[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        bias[i].x = a.bias && 2 * i < cn ? a.bias[tile.ch + c4 + 2 * i] : 0.f;
        bias[i].y = a.bias && 2 * i + 1 < cn ? a.bias[tile.ch + c4 + 2 * i + 1] : 0.f;
        skip[i].x = a.skip && 2 * i < cn ? a.skip[tile.ch + c4 + 2 * i] : 0.f;
        skip[i].y = a.skip && 2 * i + 1 < cn ? a.skip[tile.ch + c4 + 2 * i + 1] : 0.f;
    }
    float2 A2[2][4], dA[2][4];
    load_thread_states(A2, a.A, 0, a, d0, end, s0, 0);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s) A2[p][s] = mul2(A2[p][s], both(kLog2e));
    // A running sum over all of a part's tokens would lose bits: dA, d skip and d bias are summed over a block in registers, and
    // added up over the part's blocks in global memory (each word by one thread alone, with nothing to wait for) and in sm.ch.
    sm.ch[0][tid] = sm.ch[1][tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    bool kept = false;

    const int64_t slots = slots_for(a.T, a.N, kShift);
    for (int64_t slot = part; slot < slots; slot += a.parts) {
        const SeqBlock blk = find_slot(a, kShift, slot);
        if (blk.seq < 0 || blk.count == 0) continue;  // the same for the whole CTA
        typedef Rows<X, kTile, kThreads, kSub> RowsOf;
        typedef Rows<X, kSP, kThreads, kSub> StatesOf;
        auto load = [&](int buf, int t) {
            if (t >= 0) {
                const int rows = blk.count - t;
                const int64_t at = blk.start;
                RowsOf(a.x, at * a.x_st + tile.ch, a.x_st, tile.n, a.vec).stage(sm.rows[buf][0], t, rows);
                RowsOf(a.dt, at * a.dt_st + tile.ch, a.dt_st, tile.n, a.vec).stage(sm.rows[buf][1], t, rows);
                RowsOf(a.dy, at * a.dy_st + tile.ch, a.dy_st, tile.n, a.vec).stage(sm.rows[buf][2], t, rows);
                if (kGate) RowsOf(a.z, at * a.z_st + tile.ch, a.z_st, tile.n, a.vec).stage(sm.rows[buf][3], t, rows);
                StatesOf(a.b, at * a.b_st + tile.group * a.b_sg, a.b_st, a.S, a.vec).stage(sm.states[buf][0], t, rows);
                StatesOf(a.c, at * a.c_st + tile.group * a.c_sg, a.c_st, a.S, a.vec).stage(sm.states[buf][1], t, rows);
            }
            cp_async_commit();
        };
        int t0 = (blk.count - 1) / kSub * kSub, buf = 0;
        __syncthreads();  // the last block has been finished
        load(0, t0);
        float2 g[2][4];
        load_thread_states(g, a.table, slot, a, d0, end, s0, 0);
        zero(dA);
        d_skip[0] = d_skip[1] = d_bias[0] = d_bias[1] = both(0.f);
        for (; t0 >= 0; t0 -= kSub) {
            const int n = min(kSub, blk.count - t0);
            float2 h[2][4];
            load_thread_states(h, a.ckpt, static_cast<int64_t>(blk.first) / kSave + blk.seq + (blk.start - blk.first + t0) / kSave, a, d0, end, s0, 0);
            cp_async_wait<0>();
            __syncthreads();  // these tokens have come, and the last ones have been finished
            if (kBufs == 2) load(buf ^ 1, t0 - kSub);
            const X *xs = sm.rows[buf][0], *ds = sm.rows[buf][1], *ys = sm.rows[buf][2], *zs = sm.rows[buf][3];
            // tokens are worked on in fours: the ones beyond the last have steps, inputs and gradients of 0, which change nothing
            const int n4 = (n + 3) & ~3;
#pragma unroll
            for (int r = r4; r < kSub; r += kRows) {
                const int at = r * kTile + c4;
                if (r >= n) {
                    if (r < n4) *reinterpret_cast<float4*>(&sm.dt[r][c4]) = *reinterpret_cast<float4*>(&sm.u[r][c4]) = *reinterpret_cast<float4*>(&sm.dp[r][c4]) = make_float4(0.f, 0.f, 0.f, 0.f);
                    continue;
                }
                const float4 x = load4<X>(xs, at, 4, 1), v = load4<X>(ds, at, 4, 1), dy = load4<X>(ys, at, 4, 1);
                const float2 t0 = steps_of(add2(lo(v), bias[0]), a.softplus), t1 = steps_of(add2(hi(v), bias[1]), a.softplus);
                const float2 u0 = mul2(t0, lo(x)), u1 = mul2(t1, hi(x));
                float2 p0 = lo(dy), p1 = hi(dy);
                if (kGate) {
                    const float4 z = load4<X>(zs, at, 4, 1);
                    p0 = mul2(p0, act_fwd2<LA_ACT_SILU>(lo(z)));
                    p1 = mul2(p1, act_fwd2<LA_ACT_SILU>(hi(z)));
                }
                *reinterpret_cast<float4*>(&sm.dt[r][c4]) = make_float4(t0.x, t0.y, t1.x, t1.y);
                *reinterpret_cast<float4*>(&sm.u[r][c4]) = make_float4(u0.x, u0.y, u1.x, u1.y);
                *reinterpret_cast<float4*>(&sm.dp[r][c4]) = make_float4(p0.x, p0.y, p1.x, p1.y);
            }
            for (int i = tid; i < n4 * Q; i += kThreads) {
                const bool there = i < n * Q;
                const float4 zeros = make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(&sm.b[0][0] + 4 * i) = there ? load4<X>(sm.states[buf][0], 4 * i, 4, 1) : zeros;
                *reinterpret_cast<float4*>(&sm.c[0][0] + 4 * i) = there ? load4<X>(sm.states[buf][1], 4 * i, 4, 1) : zeros;
            }
            __syncthreads();

            // forward: the states before every fourth token, and p
#pragma unroll 1
            for (int k = 0; 4 * k < n; ++k) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    sm.h[w][k][2 * p][lane] = make_float4(h[p][0].x, h[p][0].y, h[p][1].x, h[p][1].y);
                    sm.h[w][k][2 * p + 1][lane] = make_float4(h[p][2].x, h[p][2].y, h[p][3].x, h[p][3].y);
                }
                if (!kGate && 4 * k + 4 >= n) break;
                float y[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * k + i;
                    const float4 dt = *reinterpret_cast<const float4*>(&sm.dt[r][cl]), u = *reinterpret_cast<const float4*>(&sm.u[r][cl]);
                    const float4 b = *reinterpret_cast<const float4*>(&sm.b[r][s0]), c = *reinterpret_cast<const float4*>(&sm.c[r][s0]);
                    const float bs[4] = {b.x, b.y, b.z, b.w}, cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 d2 = p ? hi(dt) : lo(dt), u2 = p ? hi(u) : lo(u);
                        float2 v;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float2 l = fma2(d2, A2[p][s], both(kEx2Low));
                            h[p][s] = fma2(make_float2(ex2(l.x), ex2(l.y)), h[p][s], mul2(u2, both(bs[s])));
                            if (kGate) v = s ? fma2(h[p][s], both(cs[s]), v) : mul2(h[p][s], both(cs[s]));
                        }
                        y[i][2 * p] = v.x;
                        y[i][2 * p + 1] = v.y;
                    }
                }
                if (kGate) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = spread_sum<4, 1, Q>(y[i]);
                        if (q < 4) sm.r[4 * k + i][cl + at] = y[i][0];
                    }
                }
            }
            if (kGate) {  // dz = dy p silu'(z)
                __syncthreads();
#pragma unroll
                for (int r = r4; r < kSub; r += kRows) {
                    if (r >= n) break;
                    const int at = r * kTile + c4;
                    const float4 x = load4<X>(xs, at, 4, 1), z = load4<X>(zs, at, 4, 1), dy = load4<X>(ys, at, 4, 1);
                    const float4 p = *reinterpret_cast<const float4*>(&sm.r[r][c4]);
                    float2 s0, s1;
                    act_grad2<LA_ACT_SILU>(lo(z), s0);
                    act_grad2<LA_ACT_SILU>(hi(z), s1);
                    s0 = mul2(mul2(lo(dy), fma2(skip[0], lo(x), lo(p))), s0);
                    s1 = mul2(mul2(hi(dy), fma2(skip[1], hi(x), hi(p))), s1);
                    store4<X>(a.dz, (blk.start + t0 + r) * a.dz_st + tile.ch + c4, cn, a.vec, make_float4(s0.x, s0.y, s1.x, s1.y));
                }
                __syncthreads();
            }

            // four tokens at a time from the end
#pragma unroll 1
            for (int k = (n - 1) / 4; k >= 0; --k) {
                float2 hs[5][2][4], al[4][2][4];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float4 h0 = sm.h[w][k][2 * p][lane], h1 = sm.h[w][k][2 * p + 1][lane];
                    hs[0][p][0] = lo(h0);
                    hs[0][p][1] = hi(h0);
                    hs[0][p][2] = lo(h1);
                    hs[0][p][3] = hi(h1);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * k + i;
                    const float4 dt = *reinterpret_cast<const float4*>(&sm.dt[r][cl]), u = *reinterpret_cast<const float4*>(&sm.u[r][cl]);
                    const float4 b = *reinterpret_cast<const float4*>(&sm.b[r][s0]);
                    const float bs[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 d2 = p ? hi(dt) : lo(dt), u2 = p ? hi(u) : lo(u);
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float2 l = fma2(d2, A2[p][s], both(kEx2Low));
                            al[i][p][s] = make_float2(ex2(l.x), ex2(l.y));
                            hs[i + 1][p][s] = fma2(al[i][p][s], hs[i][p][s], mul2(u2, both(bs[s])));
                        }
                    }
                }
                // what a token takes from shared memory: requested before the sums of the one after it go over the lanes
                // (what is written between would hold the reads back)
                float4 dt, u, dp, b, c;
                auto fetch = [&](int r) {
                    dt = *reinterpret_cast<const float4*>(&sm.dt[r][cl]);
                    u = *reinterpret_cast<const float4*>(&sm.u[r][cl]);
                    dp = *reinterpret_cast<const float4*>(&sm.dp[r][cl]);
                    b = *reinterpret_cast<const float4*>(&sm.b[r][s0]);
                    c = *reinterpret_cast<const float4*>(&sm.c[r][s0]);
                };
                fetch(4 * k + 3);
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    const int r = 4 * k + i;
                    const float bs[4] = {b.x, b.y, b.z, b.w}, cs[4] = {c.x, c.y, c.z, c.w};
                    float2 db[4], dc[4];
                    float t[8];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 d2 = p ? hi(dt) : lo(dt), u2 = p ? hi(u) : lo(u), p2 = p ? hi(dp) : lo(dp);
                        float2 du, wa;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float2 e = fma2(p2, both(cs[s]), g[p][s]);
                            db[s] = p ? fma2(e, u2, db[s]) : mul2(e, u2);
                            dc[s] = p ? fma2(p2, hs[i + 1][p][s], dc[s]) : mul2(p2, hs[i + 1][p][s]);
                            du = s ? fma2(e, both(bs[s]), du) : mul2(e, both(bs[s]));
                            g[p][s] = mul2(al[i][p][s], e);
                            const float2 ww = mul2(g[p][s], hs[i][p][s]);
                            wa = s ? fma2(ww, A2[p][s], wa) : mul2(ww, A2[p][s]);
                            dA[p][s] = fma2(ww, d2, dA[p][s]);
                        }
                        t[2 * p] = du.x;
                        t[2 * p + 1] = du.y;
                        t[4 + 2 * p] = wa.x;
                        t[5 + 2 * p] = wa.y;
                    }
                    if (i > 0) fetch(r - 1);
                    float v[8];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        v[s] = db[s].x + db[s].y;
                        v[4 + s] = dc[s].x + dc[s].y;
                    }
                    // over the warp's channels: value number at.. of dB (four states), dC (four states)
                    const int at = spread_sum<8, Q, 32>(v);
                    constexpr int kLeft = 32 / Q >= 8 ? 1 : 8 * Q / 32;
#pragma unroll
                    for (int j = 0; j < kLeft; ++j) sm.dbc[w][r][(at + j) / 4 * kSP + s0 + (at + j) % 4] = v[j];
                    // over the channels' states: du, then w A; every lane has read its u before it takes part
                    const int to = spread_sum<8, 1, Q>(t);
                    constexpr int kHave = Q >= 8 ? 1 : 8 / Q;
                    float* const out = to < 4 ? &sm.u[r][cl + to] : &sm.r[r][cl + to - 4];
                    if (q < 8) {
#pragma unroll
                        for (int j = 0; j < kHave; ++j) out[j] = t[j];
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = r4; r < kSub; r += kRows) {
                if (r >= n) break;
                const int at = r * kTile + c4;
                const int64_t tok = blk.start + t0 + r;
                const float4 x = load4<X>(xs, at, 4, 1), v = load4<X>(ds, at, 4, 1);
                const float4 dt = *reinterpret_cast<const float4*>(&sm.dt[r][c4]), du = *reinterpret_cast<const float4*>(&sm.u[r][c4]);
                const float4 dp = *reinterpret_cast<const float4*>(&sm.dp[r][c4]), wa = *reinterpret_cast<const float4*>(&sm.r[r][c4]);
                constexpr float kLn2 = 0.6931471805599453f;
                float2 o[2], dd[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 x2 = p ? hi(x) : lo(x), raw = add2(p ? hi(v) : lo(v), bias[p]), u2 = p ? hi(du) : lo(du), p2 = p ? hi(dp) : lo(dp);
                    o[p] = fma2(u2, p ? hi(dt) : lo(dt), mul2(p2, skip[p]));
                    dd[p] = fma2(u2, x2, mul2(p ? hi(wa) : lo(wa), both(kLn2)));
                    if (a.softplus) dd[p] = mul2(dd[p], act_fwd2<LA_ACT_SIGMOID>(raw));
                    d_skip[p] = fma2(p2, x2, d_skip[p]);
                    d_bias[p] = add2(d_bias[p], dd[p]);
                }
                store4<X>(a.dx, tok * a.dx_st + tile.ch + c4, cn, a.vec, make_float4(o[0].x, o[0].y, o[1].x, o[1].y));
                store4<X>(a.ddt, tok * a.ddt_st + tile.ch + c4, cn, a.vec, make_float4(dd[0].x, dd[0].y, dd[1].x, dd[1].y));
            }
            for (int i = tid; i < n * 2 * kSP; i += kThreads) {
                const int r = i / (2 * kSP), j = i % (2 * kSP), s = j % kSP;
                if (s >= a.S) continue;
                float v = sm.dbc[0][r][j];
#pragma unroll
                for (int k = 1; k < kWarps; ++k) v += sm.dbc[k][r][j];
                const int64_t at = (static_cast<int64_t>(tl - tile.group * a.tiles_pg) * a.T + blk.start + t0 + r) * a.G + tile.group;
                a.dbc[(at * 2 + j / kSP) * a.S + s] = v;
            }
            if (kBufs == 1) {
                __syncthreads();
                load(0, t0 - kSub);
            } else {
                buf ^= 1;
            }
        }
        if (kept) add_thread_states(dA, a.pA, part, a, d0, end, s0);
        else store_thread_states(dA, a.pA, part, a, d0, end, s0, 0);
        kept = true;
        add4(sm.ch[0][tid], d_skip);
        add4(sm.ch[1][tid], d_bias);
    }
    if (!kept) {
        zero(dA);
        store_thread_states(dA, a.pA, part, a, d0, end, s0, 0);
    }
    // d skip and d bias over the threads that share their channels, in order
    cp_async_wait<0>();
    __syncthreads();
    for (int i = tid; i < 2 * kTile; i += kThreads) {
        const int which = i / kTile, c = i % kTile;
        if (c >= tile.n) continue;
        const float* from = reinterpret_cast<const float*>(&sm.ch[which][0]) + c;  // [kRows][kTile]
        float t = 0.f;
        for (int r = 0; r < kRows; ++r) t += from[r * kTile];
        a.pch[(static_cast<int64_t>(part) * 2 + which) * a.D + tile.ch + c] = t;
    }
}

// ---------------------------------------------------------------- sums over tiles and parts
// p[0] + p[pitch] + ... over `rows` rows as eight sums, of every eighth row, and pairs of those: up to 304 parts would cost a
// single running sum its last bits.
__device__ __forceinline__ float sum_in_eight(const float* p, int64_t pitch, int rows) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = i < rows ? p[i * pitch] : 0.f;
    for (int r = 8; r < rows; r += 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += r + i < rows ? p[(r + i) * pitch] : 0.f;
#pragma unroll
    for (int n = 1; n < 8; n *= 2)
#pragma unroll
        for (int i = 0; i < 8; i += 2 * n) s[i] += s[i + n];
    return s[0];
}
template <typename X>
__global__ void __launch_bounds__(256) ssm_sum_bc_kernel(const Args a) {
    const int64_t e = blockIdx.x * 256ll + threadIdx.x, n = a.T * a.G * 2 * a.S;
    if (e >= n) return;
    const float t = sum_in_eight(a.dbc + e, n, a.tiles_pg);
    const int64_t row = e / (2 * a.S), j = e - row * 2 * a.S;
    X* to = static_cast<X*>(j < a.S ? a.db : a.dc);
    to[row * a.S + (j < a.S ? j : j - a.S)] = from_f<X>(t);
}
__global__ void __launch_bounds__(256) ssm_sum_parts_kernel(const Args a) {
    const int64_t e = blockIdx.x * 256ll + threadIdx.x, DS = static_cast<int64_t>(a.D) * a.S;
    if (e < DS) {
        a.dA[e] = sum_in_eight(a.pA + e, DS, a.parts);
    } else if (e < DS + 2 * a.D) {
        const int64_t c = e - DS;
        float* to = c < a.D ? a.dskip : a.dbias;
        if (to) to[c < a.D ? c : c - a.D] = sum_in_eight(a.pch + c, 2 * a.D, a.parts);
    }
}

template <typename X, int kS, int Q>
void block_gradients(Args a, cudaStream_t s) {
    constexpr int kW = Stage<X, kS, Q>::kW;
    a.tiles_pg = (a.Dg + kW - 1) / kW;
    const dim3 grid = slot_grid(a.tiles_pg * a.G, slots_for(a.T, a.N, kShift));
    if (a.z) ssm_block_gradient_kernel<X, kS, Q, true><<<grid, 32, 0, s>>>(a);
    else ssm_block_gradient_kernel<X, kS, Q, false><<<grid, 32, 0, s>>>(a);
}

template <typename X, int Q, bool kGate>
la_status blocks(Args& a, cudaStream_t s) {
    constexpr int kTile = Work<X, Q>::kTile, kSmem = sizeof(Work<X, Q>);
    a.tiles_pg = (a.Dg + kTile - 1) / kTile;
    if (cudaFuncSetAttribute(ssm_block_kernel<X, Q, kGate>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LA_ERR_CUDA;
    }
    ssm_block_kernel<X, Q, kGate><<<static_cast<unsigned>(a.parts * a.tiles_pg * a.G), kThreads, kSmem, s>>>(a);
    return LA_OK;
}

template <typename X>
la_status run(Args& a, cudaStream_t s) {
    if (a.N > 0) {
        if (a.T > 0) {
            if (a.S <= 8) block_gradients<X, 8, 1>(a, s);
            else if (a.S <= 16) block_gradients<X, 16, 1>(a, s);
            else if (a.S <= 32) block_gradients<X, 16, 2>(a, s);
            else block_gradients<X, 16, 4>(a, s);
        }
        const unsigned bx = static_cast<unsigned>((static_cast<int64_t>(a.D) * a.S + 127) / 128);
        ssm_join_back_kernel<<<slot_grid(static_cast<int>(bx), a.N), 128, 0, s>>>(a);
    }
    la_status st;
    if (a.S <= 16) st = a.z ? blocks<X, 4, true>(a, s) : blocks<X, 4, false>(a, s);
    else if (a.S <= 32) st = a.z ? blocks<X, 8, true>(a, s) : blocks<X, 8, false>(a, s);
    else st = a.z ? blocks<X, 16, true>(a, s) : blocks<X, 16, false>(a, s);
    if (st != LA_OK) return st;
    const int64_t n = a.T * a.G * 2 * a.S;
    if (n > 0) ssm_sum_bc_kernel<X><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a);
    ssm_sum_parts_kernel<<<static_cast<unsigned>((static_cast<int64_t>(a.D) * a.S + 2 * a.D + 255) / 256), 256, 0, s>>>(a);
    return launched();
}

}  // namespace

int bwd_width(int S) { return kWarps * (S <= 16 ? 32 : S <= 32 ? 16 : 8); }
int64_t bwd_blocks(int64_t T, int32_t N) { return slots_for(T, N, kShift); }

// How many CTAs share a tile's blocks: enough to fill the GPU two to an SM, none without a block.
int bwd_parts(int64_t T, int32_t N, int D, int S, int G) {
    const int width = bwd_width(S);
    const int64_t tiles = static_cast<int64_t>((D / G + width - 1) / width) * G;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(bwd_blocks(T, N), (2 * kSms + tiles - 1) / tiles)));
}

la_status run_bwd(Args a, int32_t dtype, cudaStream_t s) { return dtype == LA_DTYPE_BF16 ? run<bf16>(a, s) : run<float>(a, s); }

}  // namespace ssm
}  // namespace la
