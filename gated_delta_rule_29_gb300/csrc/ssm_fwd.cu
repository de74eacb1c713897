// ssm_fwd.cu -- the selective scan's forward (ssm.cuh has the formulas).
//
// A warp takes 128 / Q channels of one time block and walks its tokens, some at a time through shared memory: rows by
// cp.async one stage ahead, then the steps and dt x in 32 bits, then the tokens, whose sums over the states replace
// dt x, then the skip, the gate and the store.
//
// Time is split where the channels of all sequences are too few to fill the GPU: blocks of 2^shift tokens from each sequence's start.
// A first launch leaves what each block but the last makes of a zero state, and its steps' sum; a second one goes along
// each sequence, state = e^(A sum) state + that; the main launch then starts from what enters its block.
#include "ssm.cuh"

namespace la {
namespace ssm {
namespace {

__device__ __forceinline__ void cp_async16(void* s, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <typename X, int Q>
struct Stage {
    static constexpr int kW = 128 / Q;                                       // channels of a warp
    static constexpr int kTok = Q == 1 ? 8 : Q == 2 || Q == 16 ? 16 : 32;    // tokens of a stage; divides kSave
    static constexpr int kVec = 16 / static_cast<int>(sizeof(X));
    static constexpr int kSB = 4 * Q > kVec ? 4 * Q : kVec;                  // states, padded to a wide access
    X rows[2][3][kTok * kW];    // x, dt, z
    X states[2][2][kTok * kSB]; // B, C
    float dt[kTok * kW], u[kTok * kW];
    float b[kTok * 4 * Q], c[kTok * 4 * Q];
};

// Rows [0, rows) of n elements into shared memory, padded with zeros to kWidth.
template <typename X, int kWidth>
__device__ __forceinline__ void stage_rows(X* s, const void* base, int64_t at, int64_t stride, int rows, int n, int vec) {
    constexpr int kVec = 16 / static_cast<int>(sizeof(X)), kVecs = kWidth / kVec;
    const X* g = static_cast<const X*>(base) + at;
    for (int i = threadIdx.x & 31; i < rows * kVecs; i += 32) {
        const int r = i / kVecs, c = i % kVecs * kVec;
        const X* p = g + r * stride + c;
        if (vec && c + kVec <= n) cp_async16(s + r * kWidth + c, p);
        else
#pragma unroll
            for (int e = 0; e < kVec; ++e) s[r * kWidth + c + e] = c + e < n ? p[e] : from_f<X>(0.f);
    }
}

template <typename X, int Q, bool kLocal>
__global__ void __launch_bounds__(32) ssm_scan_kernel(const Args a) {
    typedef Stage<X, Q> Sm;
    constexpr int kW = Sm::kW, kTok = Sm::kTok, kSP = 4 * Q;
    __shared__ __align__(16) Sm sm;
    const int lane = threadIdx.x, q = lane % Q, cg = lane / Q;
    const int64_t slot = this_slot();
    if (slot >= slots_for(a.T, a.N, a.shift)) return;
    if (!kLocal && blockIdx.x == 0 && lane == 0 && slot < a.N) check_cu(a.cu, a.cu64, a.N, a.T, slot, a.status);
    const SeqBlock blk = find_time_block(a, a.shift, slot);
    if (blk.seq < 0) return;
    const bool last = blk.start + blk.count == blk.first + blk.len;
    if (kLocal && last) return;  // what the last block leaves, nobody takes over
    const Tile tile = tile_of(a, blockIdx.x, kW);
    const int d0 = tile.ch + 4 * cg, end = tile.ch + tile.n, s0 = 4 * q;

    float2 A2[2][4], h[2][4];
    load_thread_states(A2, a.A, 0, a, d0, end, s0, 0);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s) A2[p][s] = mul2(A2[p][s], both(kLog2e));
    zero(h);
    int64_t row0 = -1;
    if (!kLocal) {
        const bool split = blk.len > (int64_t(1) << a.shift);
        if (a.s0) {
            row0 = state_row(a, blk.seq);
            if (row0 < 0) return;
        }
        if (split) load_thread_states(h, a.table, slot, a, d0, end, s0, 0);
        else if (a.s0) load_thread_states(h, a.s0, row0, a, d0, end, s0, a.s0_bf16);
    }
    // the channels that this lane prepares and finishes: four of them, of every kRows-th row
    constexpr int kVecs = kW / 4, kRows = 32 / kVecs;
    const int c4 = lane % kVecs * 4, r4 = lane / kVecs;
    float bias[4], skip[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool live = c4 + i < tile.n;
        bias[i] = live && a.bias ? a.bias[tile.ch + c4 + i] : 0.f;
        skip[i] = !kLocal && live && a.skip ? a.skip[tile.ch + c4 + i] : 0.f;
    }
    float2 sum[2] = {both(0.f), both(0.f)};

    auto load = [&](int buf, int t) {
        const int n = min(kTok, blk.count - t);
        const int64_t tok = blk.start + t;
        if (n > 0) {
            stage_rows<X, kW>(sm.rows[buf][0], a.x, tok * a.x_st + tile.ch, a.x_st, n, tile.n, a.vec);
            stage_rows<X, kW>(sm.rows[buf][1], a.dt, tok * a.dt_st + tile.ch, a.dt_st, n, tile.n, a.vec);
            if (!kLocal && a.z) stage_rows<X, kW>(sm.rows[buf][2], a.z, tok * a.z_st + tile.ch, a.z_st, n, tile.n, a.vec);
            stage_rows<X, Sm::kSB>(sm.states[buf][0], a.b, tok * a.b_st + tile.group * a.b_sg, a.b_st, n, a.S, a.vec);
            if (!kLocal) stage_rows<X, Sm::kSB>(sm.states[buf][1], a.c, tok * a.c_st + tile.group * a.c_sg, a.c_st, n, a.S, a.vec);
        }
        cp_async_commit();
    };
    load(0, 0);
    int buf = 0;
    for (int t0 = 0; t0 < blk.count; t0 += kTok, buf ^= 1) {
        load(buf ^ 1, t0 + kTok);
        cp_async_wait<1>();
        __syncwarp();
        const int n = min(kTok, blk.count - t0);
        for (int r = r4; r < n; r += kRows) {
            const float4 x = load4<X>(sm.rows[buf][0], r * kW + c4, 4, 1), raw = load4<X>(sm.rows[buf][1], r * kW + c4, 4, 1);
            const float4 dt = make_float4(step_of(raw.x + bias[0], a.softplus), step_of(raw.y + bias[1], a.softplus),
                                          step_of(raw.z + bias[2], a.softplus), step_of(raw.w + bias[3], a.softplus));
            *reinterpret_cast<float4*>(sm.dt + r * kW + c4) = dt;
            *reinterpret_cast<float4*>(sm.u + r * kW + c4) = make_float4(dt.x * x.x, dt.y * x.y, dt.z * x.z, dt.w * x.w);
        }
        for (int i = lane; i < n * kSP; i += 32) {
            const int r = i / kSP, s = i % kSP;
            sm.b[i] = to_f(sm.states[buf][0][r * Sm::kSB + s]);
            if (!kLocal) sm.c[i] = to_f(sm.states[buf][1][r * Sm::kSB + s]);
        }
        __syncwarp();
        if (!kLocal && a.ckpt && t0 % kSave == 0) {
            const int64_t at = (static_cast<int64_t>(blk.first) / kSave) + blk.seq + (blk.start - blk.first + t0) / kSave;
            store_thread_states(h, a.ckpt, at, a, d0, end, s0, 0);
        }
#pragma unroll 2
        for (int r = 0; r < n; ++r) {
            const float4 dt = *reinterpret_cast<const float4*>(sm.dt + r * kW + 4 * cg), u = *reinterpret_cast<const float4*>(sm.u + r * kW + 4 * cg);
            const float4 b = *reinterpret_cast<const float4*>(sm.b + r * kSP + s0);
            const float bs[4] = {b.x, b.y, b.z, b.w};
            float4 c;
            if (!kLocal) c = *reinterpret_cast<const float4*>(sm.c + r * kSP + s0);
            const float cs[4] = {c.x, c.y, c.z, c.w};
            float v[4];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 dp = p ? hi(dt) : lo(dt), up = p ? hi(u) : lo(u);
                float2 y;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float2 l = fma2(dp, A2[p][s], both(kEx2Low));
                    h[p][s] = fma2(make_float2(ex2(l.x), ex2(l.y)), h[p][s], mul2(up, both(bs[s])));
                    if (!kLocal) y = s ? fma2(h[p][s], both(cs[s]), y) : mul2(h[p][s], both(cs[s]));
                }
                if (kLocal) sum[p] = add2(sum[p], dp);
                v[2 * p] = y.x;
                v[2 * p + 1] = y.y;
            }
            if (!kLocal) {
                // every lane has read its u before it takes part in the sum that one of them writes over it
                const int at = spread_sum<4, 1, Q>(v);
                if (Q <= 4 || q < 4) {
#pragma unroll
                    for (int i = 0; i < (Q >= 4 ? 1 : 4 / Q); ++i) sm.u[r * kW + 4 * cg + at + i] = v[i];
                }
            }
        }
        __syncwarp();
        if (!kLocal && a.y) {
            for (int r = r4; r < n; r += kRows) {
                const float4 p = *reinterpret_cast<const float4*>(sm.u + r * kW + c4), x = load4<X>(sm.rows[buf][0], r * kW + c4, 4, 1);
                float2 y0 = fma2(make_float2(skip[0], skip[1]), lo(x), lo(p)), y1 = fma2(make_float2(skip[2], skip[3]), hi(x), hi(p));
                if (a.z) {
                    const float4 z = load4<X>(sm.rows[buf][2], r * kW + c4, 4, 1);
                    y0 = mul2(y0, act_fwd2<LA_ACT_SILU>(lo(z)));
                    y1 = mul2(y1, act_fwd2<LA_ACT_SILU>(hi(z)));
                }
                store4<X>(a.y, (blk.start + t0 + r) * a.y_st + tile.ch + c4, tile.n - c4, a.vec, make_float4(y0.x, y0.y, y1.x, y1.y));
            }
            __syncwarp();
        }
    }
    if (kLocal) {
        store_thread_states(h, a.table, slot, a, d0, end, s0, 0);
        if (q == 0) {
            const float v[4] = {sum[0].x, sum[0].y, sum[1].x, sum[1].y};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (d0 + i < end) a.sums[slot * a.D + d0 + i] = v[i];
        }
        return;
    }
    if (!last) return;
    if (a.idx) store_thread_states(h, const_cast<void*>(a.s0), row0, a, d0, end, s0, a.s0_bf16);
    else if (a.fin) store_thread_states(h, a.fin, blk.seq, a, d0, end, s0, 0);
}

// Along each split sequence: what its blocks make of nothing becomes what enters them.
__global__ void __launch_bounds__(128) ssm_join_kernel(const Args a) {
    const int64_t e = blockIdx.x * 128ll + threadIdx.x, DS = static_cast<int64_t>(a.D) * a.S;
    const int64_t i = this_slot();
    if (i >= a.N || e >= DS) return;
    const int64_t t0 = cu_load(a.cu, a.cu64, i), t1 = cu_load(a.cu, a.cu64, i + 1);
    if (t0 < 0 || t1 < t0 || t1 > a.T || t1 - t0 <= (int64_t(1) << a.shift)) return;
    const int64_t blocks = (t1 - t0 - 1 >> a.shift) + 1, slot = (t0 >> a.shift) + i;
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
            loc[k] = live ? a.table[(slot + c + k) * DS + e] : 0.f;
            sum[k] = live ? a.sums[(slot + c + k) * a.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (c + k < blocks) {
                a.table[(slot + c + k) * DS + e] = st;
                st = fmaf(ex2(A2 * sum[k]), st, loc[k]);
            }
    }
}

struct Scan {
    template <typename X, int Q>
    static la_status run(Args& a, cudaStream_t s) {
        constexpr int kW = Stage<X, Q>::kW;
        a.tiles_pg = (a.Dg + kW - 1) / kW;
        const int64_t slots = slots_for(a.T, a.N, a.shift);
        const dim3 grid = slot_grid(a.tiles_pg * a.G, slots);
        if (a.T > (int64_t(1) << a.shift)) {
            ssm_scan_kernel<X, Q, true><<<grid, 32, 0, s>>>(a);
            const unsigned bx = static_cast<unsigned>((static_cast<int64_t>(a.D) * a.S + 127) / 128);
            ssm_join_kernel<<<slot_grid(static_cast<int>(bx), a.N), 128, 0, s>>>(a);
        }
        ssm_scan_kernel<X, Q, false><<<grid, 32, 0, s>>>(a);
        return launched();
    }
};

}  // namespace

// Tokens of a time block: one warp takes a block of 128 / Q channels, and kFill of them fill an SM.
int fwd_shift(int64_t T, int D, int S, int G, int time_block) {
    int shift = 6;
    if (time_block > 0) {
        while ((1 << shift) < time_block) ++shift;
        return shift;
    }
    constexpr int kFill = 8;
    const int64_t width = 128 / lanes_for(S), tiles = (D / G + width - 1) / width * G;
    while (shift < 30 && (T * tiles >> shift) > kSms * kFill) ++shift;
    return shift;
}

la_status run_fwd(Args a, int32_t dtype, cudaStream_t s) { return by_shape<Scan>(dtype, a.S, a, s); }

}  // namespace ssm
}  // namespace la
