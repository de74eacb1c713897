// ssm_fwd.cu -- the selective scan's forward (ssm.cuh has the formulas).
//
// A warp takes 32 / Q channels of one time block and walks its tokens, 16 at a time through shared memory, the next ones
// on their way meanwhile (cp.async).  A lane has one channel with kS of its states, so that B and C are the same address for
// 32 or 16 neighbouring lanes (two cycles for 16 bytes a lane, measured, where addresses that alternate between lanes
// take four), pairs of states come as they lie, and up to 16 states no sum goes over lanes.  What two tokens' scans need
// beside B and C is formed while the two before are scanned.
//
// Bound by a warp's latency where it walks its tokens almost alone: about 350 cycles a token.  8 x 8192 x 4096 x 16 are 1024 such
// warps on 608 schedulers, and their 8192 tokens at 350 cycles are its 1.46 ms (2.9e12 state steps a second; its bytes would take
// 0.32 ms).  With schedulers full a token takes 196 cycles: 99 instructions, 43 of them pairs of fp32 operations, which take two
// slots, fill 142; the states alone, in a loop of their own, take 105.
//
// Time is split where the channels of all sequences are too few to fill the GPU: blocks of 2^shift tokens from each sequence's start.
// A first launch leaves what each block but the last makes of a zero state, and its steps' sum; a second one goes along
// each sequence, state = e^(A sum) state + that; the main launch then starts from what enters its block.
#include "ssm.cuh"

namespace la {
namespace ssm {
namespace {

constexpr int kTok = 16;  // tokens of a stage; saved states lie between stages
static_assert(kTok == kSave, "");

template <typename X, int kS, int Q>
struct Stage {
    static constexpr int kW = 32 / Q, kSP = kS * Q;  // channels of a warp, states of a channel
    X rows[2][3][kTok * kW];                         // x, dt, z
    X states[2][2][kTok * kSP];                      // B, C
    float wide[sizeof(X) == 4 ? 1 : 2][sizeof(X) == 4 ? 4 : kTok * kSP];  // B and C in 32 bits, where they are not so already
};

template <typename X, int kS, int Q, bool kLocal, bool kGate>
__global__ void __launch_bounds__(32, 14) ssm_scan_kernel(const Args a) {
    typedef Stage<X, kS, Q> Sm;
    constexpr int kW = Sm::kW, kSP = Sm::kSP, kPairs = kS / 2;
    __shared__ __align__(16) Sm sm;
    const int lane = threadIdx.x, q = lane / kW, ch = lane % kW;
    const int64_t slot = this_slot();
    if (slot >= slots_for(a.T, a.N, a.shift)) return;
    if (!kLocal && blockIdx.x == 0 && lane == 0 && slot < a.N) check_cu(a.cu, a.cu64, a.N, a.T, slot, a.status);
    const SeqBlock blk = find_launched(a, a.shift, slot);
    if (blk.seq < 0) return;
    const bool last = blk.start + blk.count == blk.first + blk.len;
    if (kLocal && last) return;  // what the last block leaves, nobody takes over
    const Tile tile = tile_of(a, blockIdx.x, kW);
    const int d = tile.ch + ch, s0 = kS * q;
    const bool live = ch < tile.n;

    typedef Rows<X, kW, 32, kTok> RowsOf;
    typedef Rows<X, kSP, 32, kTok> StatesOf;
    const RowsOf x_rows(a.x, blk.start * a.x_st + tile.ch, a.x_st, tile.n, a.vec), dt_rows(a.dt, blk.start * a.dt_st + tile.ch, a.dt_st, tile.n, a.vec),
        z_rows(a.z, blk.start * a.z_st + tile.ch, a.z_st, tile.n, a.vec);
    const StatesOf b_rows(a.b, blk.start * a.b_st + tile.group * a.b_sg, a.b_st, a.S, a.vec), c_rows(a.c, blk.start * a.c_st + tile.group * a.c_sg, a.c_st, a.S, a.vec);
    auto load = [&](int buf, int t) {
        const int rows = blk.count - t;
        x_rows.stage(sm.rows[buf][0], t, rows);
        dt_rows.stage(sm.rows[buf][1], t, rows);
        if (kGate) z_rows.stage(sm.rows[buf][2], t, rows);
        b_rows.stage(sm.states[buf][0], t, rows);
        if (!kLocal) c_rows.stage(sm.states[buf][1], t, rows);
        cp_async_commit();
    };
    load(0, 0);

    float2 A2[kPairs], h[kPairs];
    load_lane_states<kS>(A2, a.A, 0, a, d, s0, live, 0);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        A2[k] = mul2(A2[k], both(kLog2e));
        h[k] = both(0.f);
    }
    int64_t row0 = -1;
    if (!kLocal) {
        if (a.s0) {
            row0 = state_row(a, blk.seq);
            if (row0 < 0) {
                cp_async_wait<0>();
                return;
            }
        }
        if (split(blk.len, a.shift)) load_lane_states<kS>(h, a.table, slot, a, d, s0, live, 0);
        else if (a.s0) load_lane_states<kS>(h, a.s0, row0, a, d, s0, live, a.s0_bf16);
    }
    const float bias = live && a.bias ? a.bias[d] : 0.f, skip = !kLocal && live && a.skip ? a.skip[d] : 0.f;
    const bool stores = live && q == 0 && a.y;
    float sum = 0.f;
    X* out = kLocal ? nullptr : static_cast<X*>(a.y) + blk.start * a.y_st + d;

    int buf = 0;
    for (int t0 = 0; t0 < blk.count; t0 += kTok, buf ^= 1) {
        load(buf ^ 1, t0 + kTok);
        cp_async_wait<1>();
        __syncwarp();
        const int n = min(kTok, blk.count - t0);
        const float *bs, *cs;
        if constexpr (sizeof(X) == 4) {
            bs = sm.states[buf][0];
            cs = sm.states[buf][1];
        } else {
#pragma unroll
            for (int j = 0; j < kTok * kSP / 128; ++j) {  // rows beyond n hold what they held before
                const int i = 4 * (lane + 32 * j);
                *reinterpret_cast<float4*>(sm.wide[0] + i) = load4<X>(sm.states[buf][0], i, 4, 1);
                if (!kLocal) *reinterpret_cast<float4*>(sm.wide[1] + i) = load4<X>(sm.states[buf][1], i, 4, 1);
            }
            __syncwarp();
            bs = sm.wide[0];
            cs = sm.wide[1];
        }
        bs += s0;
        cs += s0;
        if (!kLocal && a.ckpt)
            store_lane_states<kS>(h, a.ckpt, static_cast<int64_t>(blk.first) / kSave + blk.seq + (blk.start - blk.first + t0) / kSave, a, d, s0, live, 0);
        const X *xs = sm.rows[buf][0] + ch, *ds = sm.rows[buf][1] + ch, *zs = sm.rows[buf][2] + ch;
        struct Pair {  // two tokens' steps, dt x, skip x and gates
            float2 dt, u, rest, gate;
        };
        // no branch within, so that the latency of its chain (some 150 cycles) is filled with the scans beside it
        auto prepare = [&](int r) {
            Pair t;
            const float2 x = make_float2(to_f(xs[r * kW]), to_f(xs[r * kW + kW])), raw = add2(make_float2(to_f(ds[r * kW]), to_f(ds[r * kW + kW])), both(bias));
            const float2 sp = softplus2(raw);
            t.dt = make_float2(a.softplus ? sp.x : raw.x, a.softplus ? sp.y : raw.y);
            t.u = mul2(t.dt, x);
            if (!kLocal) t.rest = mul2(both(skip), x);
            if (kGate) t.gate = act_fwd2<LA_ACT_SILU>(make_float2(to_f(zs[r * kW]), to_f(zs[r * kW + kW])));
            return t;
        };
        // one token; returns this lane's part of sum_s C h
        auto token = [&](float dt, float u, int r) {
            const float2 d2 = both(dt), u2 = both(u);
            float2 y0 = both(0.f), y1 = both(0.f);
#pragma unroll
            for (int k = 0; k < kPairs; k += 2) {
                const float4 b = *reinterpret_cast<const float4*>(bs + r * kSP + 2 * k);
                const float2 l0 = fma2(d2, A2[k], both(kEx2Low)), l1 = fma2(d2, A2[k + 1], both(kEx2Low));
                h[k] = fma2(make_float2(ex2(l0.x), ex2(l0.y)), h[k], mul2(u2, lo(b)));
                h[k + 1] = fma2(make_float2(ex2(l1.x), ex2(l1.y)), h[k + 1], mul2(u2, hi(b)));
                if (!kLocal) {
                    const float4 c = *reinterpret_cast<const float4*>(cs + r * kSP + 2 * k);
                    y0 = k ? fma2(h[k], lo(c), y0) : mul2(h[k], lo(c));
                    y1 = k ? fma2(h[k + 1], hi(c), y1) : mul2(h[k + 1], hi(c));
                }
            }
            y0 = add2(y0, y1);
            return y0.x + y0.y;
        };
        auto finish = [&](const Pair& t, float2 p) {
#pragma unroll
            for (int off = kW; off < 32; off *= 2) {
                p.x += __shfl_xor_sync(0xffffffffu, p.x, off);
                p.y += __shfl_xor_sync(0xffffffffu, p.y, off);
            }
            p = add2(p, t.rest);
            return kGate ? mul2(p, t.gate) : p;
        };
        // rows beyond n are prepared too, from whatever lies there, and not used
        Pair now = prepare(0);
        int r = 0;
#pragma unroll 2
        for (; r + 1 < n; r += 2) {
            const Pair next = prepare((r + 2) % kTok);
            float2 p;
            p.x = token(now.dt.x, now.u.x, r);
            p.y = token(now.dt.y, now.u.y, r + 1);
            if (kLocal) {
                sum += now.dt.x + now.dt.y;
            } else {
                p = finish(now, p);
                if (stores) {
                    out[0] = from_f<X>(p.x);
                    out[a.y_st] = from_f<X>(p.y);
                }
                out += 2 * a.y_st;
            }
            now = next;
        }
        if (r < n) {
            const float p = token(now.dt.x, now.u.x, r);
            if (kLocal) {
                sum += now.dt.x;
            } else {
                const float2 y = finish(now, both(p));
                if (stores) out[0] = from_f<X>(y.x);
            }
        }
        __syncwarp();
    }
    if (kLocal) {
        store_lane_states<kS>(h, a.table, slot, a, d, s0, live, 0);
        if (live && q == 0) a.sums[slot * a.D + d] = sum;
        return;
    }
    if (!last) return;
    if (a.idx) store_lane_states<kS>(h, const_cast<void*>(a.s0), row0, a, d, s0, live, a.s0_bf16);
    else if (a.fin) store_lane_states<kS>(h, a.fin, blk.seq, a, d, s0, live, 0);
}

// Along each split sequence: what its blocks make of nothing becomes what enters them.
__global__ void __launch_bounds__(128) ssm_join_kernel(const Args a) {
    const int64_t e = blockIdx.x * 128ll + threadIdx.x, DS = static_cast<int64_t>(a.D) * a.S;
    const int64_t i = this_slot();
    if (i >= a.N || e >= DS) return;
    const int64_t t0 = cu_load(a.cu, a.cu64, i), t1 = cu_load(a.cu, a.cu64, i + 1);
    if (t0 < 0 || t1 < t0 || t1 > a.T || !split(t1 - t0, a.shift)) return;
    const int64_t blocks = (t1 - t0 - 1 >> a.shift) + 1;
    float st = 0.f;
    if (a.s0) {
        const int64_t row = state_row(a, static_cast<int32_t>(i));
        if (row < 0) return;
        st = load_any(a.s0, row * DS + e, a.s0_bf16);
    }
    const float A2 = a.A[e] * kLog2e;
    const int64_t d = e / a.S;
    constexpr int kAhead = 8;
    for (int64_t c = 0; c < blocks; c += kAhead) {
        float loc[kAhead], sum[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool live = c + k + 1 < blocks;  // the last block has left nothing
            const int64_t row = launched_row(a, a.shift, i, t0, c + k);
            loc[k] = live ? a.table[row * DS + e] : 0.f;
            sum[k] = live ? a.sums[row * a.D + d] : 0.f;
        }
        st = walk_blocks(st, A2, sum, loc, [&](int k, float entering) {
            if (c + k < blocks) a.table[launched_row(a, a.shift, i, t0, c + k) * DS + e] = entering;
            return c + k < blocks;
        });
    }
}

template <typename X, int kS, int Q>
la_status scan(Args& a, cudaStream_t s) {
    constexpr int kW = Stage<X, kS, Q>::kW;
    a.tiles_pg = (a.Dg + kW - 1) / kW;
    const dim3 grid = slot_grid(a.tiles_pg * a.G, slots_for(a.T, a.N, a.shift));
    if (split(a.T, a.shift)) {
        ssm_scan_kernel<X, kS, Q, true, false><<<grid, 32, 0, s>>>(a);
        const unsigned bx = static_cast<unsigned>((static_cast<int64_t>(a.D) * a.S + 127) / 128);
        ssm_join_kernel<<<slot_grid(static_cast<int>(bx), a.N), 128, 0, s>>>(a);
    }
    if (a.z) ssm_scan_kernel<X, kS, Q, false, true><<<grid, 32, 0, s>>>(a);
    else ssm_scan_kernel<X, kS, Q, false, false><<<grid, 32, 0, s>>>(a);
    return launched();
}
// Channels of a warp.
int scan_width(int S) { return S <= 16 ? 32 : S <= 32 ? 16 : 8; }
template <typename X>
la_status by_scan(Args& a, cudaStream_t s) {
    if (a.S <= 8) return scan<X, 8, 1>(a, s);
    if (a.S <= 16) return scan<X, 16, 1>(a, s);
    if (a.S <= 32) return scan<X, 16, 2>(a, s);
    return scan<X, 16, 4>(a, s);
}

}  // namespace

// Tokens of a time block: a warp takes a block of scan_width channels, and kFill of them fill an SM.  Few tokens take blocks of
// 32 where that leaves SMs less than half filled: a warp's time is then the latency of its tokens (up to two blocks of them),
// but the blocks' states cost more, and the join walks them one by one (one sequence of 200 x 1024 x 16: 15.7 us, 22.0 with 64;
// 600 tokens of three, 600 x 23: 25.2, 42.6; but 1024 x 512 x 64: 38.9, 34.1; 4096 x 256 x 8: 27.4, 24.8).
int fwd_shift(int64_t T, int D, int S, int G, int time_block) {
    int shift = 6;
    if (time_block > 0) {
        while ((1 << shift) < time_block) ++shift;
        return shift;
    }
    constexpr int kFill = 24;  // 49344 x 1024 in fp32, skewed: 470 us with 24, 641 with 16, 807 with 8
    const int64_t width = scan_width(S), tiles = (D / G + width - 1) / width * G;
    if (T <= 2048 && (T * tiles >> 5) <= kSms * 10) return 5;
    while (shift < 30 && (T * tiles >> shift) > kSms * kFill) ++shift;
    return shift;
}

la_status run_fwd(Args a, int32_t dtype, cudaStream_t s) { return dtype == LA_DTYPE_BF16 ? by_scan<bf16>(a, s) : by_scan<float>(a, s); }

}  // namespace ssm
}  // namespace la
