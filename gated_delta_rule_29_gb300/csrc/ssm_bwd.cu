// ssm_bwd.cu -- the selective scan's backward (ssm.cuh has the formulas).
//
// Time is cut into chunks of 32 tokens from each sequence's start, the state entering each being the forward's
// checkpoint.  A first launch leaves what each chunk makes of a zero gradient behind it, and its steps' sum; a second one
// goes along each sequence from its end, which gives the gradient behind every chunk; then all chunks are worked on side by
// side.  Chunks are fixed by the sequence alone, so the gradients of its inputs do not depend on the batch around it.
//
// Within a chunk a warp goes forward once, leaving the states before every fourth token in shared memory (and p, for dz),
// then takes four tokens at a time from the end: forward again with states and decays kept in registers, then back.
// dB and dC are summed over a thread's channels, the warp's, the CTA's, and by a later launch over the CTAs that share a
// group; dA, d skip and d bias over a CTA's chunks and then over the CTAs, all in an order that the shape fixes.
#include "ssm.cuh"

namespace la {
namespace ssm {
namespace {

constexpr int kShift = 5;
static_assert(kSave == 1 << kShift, "the chunks are the forward's");

// dy act(z): the gradient of p.
template <typename X>
__device__ __forceinline__ float4 p_gradient(const Args& a, int64_t tok, int ch, int n) {
    float4 g = load4<X>(a.dy, tok * a.dy_st + ch, n, a.vec);
    if (!a.z) return g;
    const float4 z = load4<X>(a.z, tok * a.z_st + ch, n, a.vec);
    const float2 s0 = mul2(lo(g), act_fwd2<LA_ACT_SILU>(lo(z))), s1 = mul2(hi(g), act_fwd2<LA_ACT_SILU>(hi(z)));
    return make_float4(s0.x, s0.y, s1.x, s1.y);
}
template <typename X>
__device__ __forceinline__ float4 raw_steps(const Args& a, int64_t tok, int ch, int n, const float (&bias)[4]) {
    const float4 r = load4<X>(a.dt, tok * a.dt_st + ch, n, a.vec);
    return make_float4(r.x + bias[0], r.y + bias[1], r.z + bias[2], r.w + bias[3]);
}
__device__ __forceinline__ float4 steps_of(float4 r, int softplus) {
    const float2 a = ssm::steps_of(lo(r), softplus), b = ssm::steps_of(hi(r), softplus);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void load_channels(float (&v)[4], const float* p, int ch, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p && i < n ? p[ch + i] : 0.f;
}

// ---------------------------------------------------------------- the gradient behind each chunk
template <typename X, int Q>
__global__ void __launch_bounds__(32) ssm_chunk_gradient_kernel(const Args a) {
    constexpr int kW = 128 / Q, kSP = 4 * Q;
    __shared__ __align__(16) float s_dt[kSave * kW], s_dp[kSave * kW], s_c[kSave * kSP];
    const int lane = threadIdx.x, q = lane % Q, cg = lane / Q;
    const int64_t slot = this_slot();
    if (slot >= slots_for(a.T, a.N, kShift)) return;
    const SeqBlock blk = find_slot(a, kShift, slot);
    if (blk.seq < 0 || blk.count == 0) return;
    const Tile tile = tile_of(a, blockIdx.x, kW);
    const int d0 = tile.ch + 4 * cg, end = tile.ch + tile.n, s0 = 4 * q;
    constexpr int kVecs = kW / 4, kRows = 32 / kVecs;
    const int c4 = lane % kVecs * 4, r4 = lane / kVecs;
    float bias[4];
    load_channels(bias, a.bias, tile.ch + c4, tile.n - c4);
#pragma unroll 4
    for (int r = r4; r < blk.count; r += kRows) {
        const int64_t tok = blk.start + r;
        *reinterpret_cast<float4*>(s_dt + r * kW + c4) = steps_of(raw_steps<X>(a, tok, tile.ch + c4, tile.n - c4, bias), a.softplus);
        *reinterpret_cast<float4*>(s_dp + r * kW + c4) = p_gradient<X>(a, tok, tile.ch + c4, tile.n - c4);
    }
    for (int i = lane; i < blk.count * Q; i += 32) {
        const int r = i / Q, s = i % Q * 4;
        *reinterpret_cast<float4*>(s_c + r * kSP + s) = load4<X>(a.c, (blk.start + r) * a.c_st + tile.group * a.c_sg + s, a.S - s, a.vec);
    }
    float2 A2[2][4], g[2][4], sum[2] = {both(0.f), both(0.f)};
    load_thread_states(A2, a.A, 0, a, d0, end, s0, 0);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s) A2[p][s] = mul2(A2[p][s], both(kLog2e));
    zero(g);
    __syncwarp();
#pragma unroll 2
    for (int r = blk.count - 1; r >= 0; --r) {
        const float4 dt = *reinterpret_cast<const float4*>(s_dt + r * kW + 4 * cg), dp = *reinterpret_cast<const float4*>(s_dp + r * kW + 4 * cg);
        const float4 c = *reinterpret_cast<const float4*>(s_c + r * kSP + s0);
        const float cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float2 t = p ? hi(dt) : lo(dt), e = p ? hi(dp) : lo(dp);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float2 l = fma2(t, A2[p][s], both(kEx2Low));
                g[p][s] = mul2(make_float2(ex2(l.x), ex2(l.y)), fma2(e, both(cs[s]), g[p][s]));
            }
            sum[p] = add2(sum[p], t);
        }
    }
    store_thread_states(g, a.table, slot, a, d0, end, s0, 0);
    if (q == 0) {
        const float v[4] = {sum[0].x, sum[0].y, sum[1].x, sum[1].y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d0 + i < end) a.sums[slot * a.D + d0 + i] = v[i];
    }
}

__global__ void __launch_bounds__(128) ssm_join_back_kernel(const Args a) {
    const int64_t e = blockIdx.x * 128ll + threadIdx.x, DS = static_cast<int64_t>(a.D) * a.S;
    const int64_t i = this_slot();
    if (i >= a.N || e >= DS) return;
    const int64_t t0 = cu_load(a.cu, a.cu64, i), t1 = cu_load(a.cu, a.cu64, i + 1);
    if (blockIdx.x == 0 && threadIdx.x == 0) check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
    if (t0 < 0 || t1 < t0 || t1 > a.T) return;
    const int64_t blocks = (t1 - t0 + kSave - 1) >> kShift, slot = (t0 >> kShift) + i;
    float g = a.dfin ? a.dfin[i * DS + e] : 0.f;
    const float A2 = a.A[e] * kLog2e;
    const int64_t d = e / a.S;
    constexpr int kAhead = 8;
    for (int64_t c = blocks - 1; c >= 0; c -= kAhead) {
        float loc[kAhead], sum[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            loc[k] = c >= k ? a.table[(slot + c - k) * DS + e] : 0.f;
            sum[k] = c >= k ? a.sums[(slot + c - k) * a.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (c >= k) {
                a.table[(slot + c - k) * DS + e] = g;
                g = fmaf(ex2(A2 * sum[k]), g, loc[k]);
            }
    }
    if (a.ds0) a.ds0[i * DS + e] = g;
}

// ---------------------------------------------------------------- all gradients of a chunk
constexpr int kWarps = 4, kThreads = 32 * kWarps;

template <int Q>
struct Work {
    static constexpr int kW = 64 / Q, kTile = kWarps * kW, kSP = 4 * Q;  // channels of a warp, of a CTA; states
    float dt[kSave][kTile], u[kSave][kTile], dp[kSave][kTile], r[kSave][kTile];  // r: p, then the sum of w A log2(e)
    float b[kSave][kSP], c[kSave][kSP];
    float4 h[kWarps][kSave / 4][2][32];   // the states before every fourth token
    float dbc[kWarps][kSave][2 * kSP];    // dB, dC of a warp's channels
};

template <typename X, int Q>
__global__ void __launch_bounds__(kThreads, 3) ssm_chunk_kernel(const Args a) {
    typedef Work<Q> Wk;
    constexpr int kW = Wk::kW, kTile = Wk::kTile, kSP = Wk::kSP;
    extern __shared__ __align__(16) uint8_t raw_smem[];
    Wk& sm = *reinterpret_cast<Wk*>(raw_smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, q = lane % Q, cg = lane / Q;
    const int tiles = a.tiles_pg * a.G, part = blockIdx.x / tiles, tl = blockIdx.x - part * tiles;
    const Tile tile = tile_of(a, tl, kTile);
    const int cl = w * kW + 2 * cg;  // the thread's first channel within the tile
    const int d0 = tile.ch + cl, end = tile.ch + tile.n, s0 = 4 * q;
    // the four channels that this thread loads and stores, of every kRows-th row
    constexpr int kVecs = kTile / 4, kRows = kThreads / kVecs;
    const int c4 = tid % kVecs * 4, r4 = tid / kVecs, cn = tile.n - c4;
    float bias[4], skip[4], d_skip[4] = {0.f, 0.f, 0.f, 0.f}, d_bias[4] = {0.f, 0.f, 0.f, 0.f};
    load_channels(bias, a.bias, tile.ch + c4, cn);
    load_channels(skip, a.skip, tile.ch + c4, cn);

    float2 A2[1][4], dA[1][4];
    load_thread_states(A2, a.A, 0, a, d0, end, s0, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) A2[0][s] = mul2(A2[0][s], both(kLog2e));
    zero(dA);

    const int64_t slots = slots_for(a.T, a.N, kShift);
    for (int64_t slot = part; slot < slots; slot += a.parts) {
        const SeqBlock blk = find_slot(a, kShift, slot);
        if (blk.seq < 0 || blk.count == 0) continue;  // the same for the whole CTA
        const int n = blk.count;
        __syncthreads();  // the last chunk's sums have been read
        for (int r = r4; r < n; r += kRows) {
            const int64_t tok = blk.start + r;
            const float4 x = load4<X>(a.x, tok * a.x_st + tile.ch + c4, cn, a.vec);
            const float4 dt = steps_of(raw_steps<X>(a, tok, tile.ch + c4, cn, bias), a.softplus);
            *reinterpret_cast<float4*>(&sm.dt[r][c4]) = dt;
            *reinterpret_cast<float4*>(&sm.u[r][c4]) = make_float4(dt.x * x.x, dt.y * x.y, dt.z * x.z, dt.w * x.w);
            *reinterpret_cast<float4*>(&sm.dp[r][c4]) = p_gradient<X>(a, tok, tile.ch + c4, cn);
        }
        for (int i = tid; i < n * Q; i += kThreads) {
            const int r = i / Q, s = i % Q * 4;
            const int64_t tok = blk.start + r;
            *reinterpret_cast<float4*>(&sm.b[r][s]) = load4<X>(a.b, tok * a.b_st + tile.group * a.b_sg + s, a.S - s, a.vec);
            *reinterpret_cast<float4*>(&sm.c[r][s]) = load4<X>(a.c, tok * a.c_st + tile.group * a.c_sg + s, a.S - s, a.vec);
        }
        float2 h[1][4], g[1][4];
        load_thread_states(h, a.ckpt, slot, a, d0, end, s0, 0);
        load_thread_states(g, a.table, slot, a, d0, end, s0, 0);
        __syncthreads();

        // forward: the states before every fourth token, and p
        for (int r = 0; r < n; ++r) {
            if (r % 4 == 0) {
                sm.h[w][r / 4][0][lane] = make_float4(h[0][0].x, h[0][0].y, h[0][1].x, h[0][1].y);
                sm.h[w][r / 4][1][lane] = make_float4(h[0][2].x, h[0][2].y, h[0][3].x, h[0][3].y);
            }
            const float2 dt = *reinterpret_cast<const float2*>(&sm.dt[r][cl]), u = *reinterpret_cast<const float2*>(&sm.u[r][cl]);
            const float4 b = *reinterpret_cast<const float4*>(&sm.b[r][s0]), c = *reinterpret_cast<const float4*>(&sm.c[r][s0]);
            const float bs[4] = {b.x, b.y, b.z, b.w}, cs[4] = {c.x, c.y, c.z, c.w};
            float2 y;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float2 l = fma2(dt, A2[0][s], both(kEx2Low));
                h[0][s] = fma2(make_float2(ex2(l.x), ex2(l.y)), h[0][s], mul2(u, both(bs[s])));
                y = s ? fma2(h[0][s], both(cs[s]), y) : mul2(h[0][s], both(cs[s]));
            }
            if (a.z) {
                float v[2] = {y.x, y.y};
                const int at = spread_sum<2, 1, Q>(v);
                if (Q == 1) *reinterpret_cast<float2*>(&sm.r[r][cl]) = make_float2(v[0], v[1]);
                else if (q < 2) sm.r[r][cl + at] = v[0];
            }
        }
        if (a.z) {  // dz = dy p silu'(z)
            __syncthreads();
            for (int r = r4; r < n; r += kRows) {
                const int64_t tok = blk.start + r;
                const float4 x = load4<X>(a.x, tok * a.x_st + tile.ch + c4, cn, a.vec), z = load4<X>(a.z, tok * a.z_st + tile.ch + c4, cn, a.vec);
                const float4 dy = load4<X>(a.dy, tok * a.dy_st + tile.ch + c4, cn, a.vec), p = *reinterpret_cast<const float4*>(&sm.r[r][c4]);
                const float2 p0 = fma2(make_float2(skip[0], skip[1]), lo(x), lo(p)), p1 = fma2(make_float2(skip[2], skip[3]), hi(x), hi(p));
                float2 t0, t1;
                act_grad2<LA_ACT_SILU>(lo(z), t0);
                act_grad2<LA_ACT_SILU>(hi(z), t1);
                t0 = mul2(mul2(lo(dy), p0), t0);
                t1 = mul2(mul2(hi(dy), p1), t1);
                store4<X>(a.dz, tok * a.dz_st + tile.ch + c4, cn, a.vec, make_float4(t0.x, t0.y, t1.x, t1.y));
            }
            __syncthreads();
        }

        // four tokens at a time from the end
        for (int k = (n - 1) / 4; k >= 0; --k) {
            float2 hs[5][4], al[4][4];
            const float4 h0 = sm.h[w][k][0][lane], h1 = sm.h[w][k][1][lane];
            hs[0][0] = lo(h0);
            hs[0][1] = hi(h0);
            hs[0][2] = lo(h1);
            hs[0][3] = hi(h1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = min(4 * k + i, n - 1);
                const float2 dt = *reinterpret_cast<const float2*>(&sm.dt[r][cl]), u = *reinterpret_cast<const float2*>(&sm.u[r][cl]);
                const float4 b = *reinterpret_cast<const float4*>(&sm.b[r][s0]);
                const float bs[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float2 l = fma2(dt, A2[0][s], both(kEx2Low));
                    al[i][s] = make_float2(ex2(l.x), ex2(l.y));
                    hs[i + 1][s] = fma2(al[i][s], hs[i][s], mul2(u, both(bs[s])));
                }
            }
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                const int r = 4 * k + i;
                if (r >= n) continue;  // the same for the whole CTA
                const float2 dt = *reinterpret_cast<const float2*>(&sm.dt[r][cl]), u = *reinterpret_cast<const float2*>(&sm.u[r][cl]);
                const float2 dp = *reinterpret_cast<const float2*>(&sm.dp[r][cl]);
                const float4 b = *reinterpret_cast<const float4*>(&sm.b[r][s0]), c = *reinterpret_cast<const float4*>(&sm.c[r][s0]);
                const float bs[4] = {b.x, b.y, b.z, b.w}, cs[4] = {c.x, c.y, c.z, c.w};
                float2 du = both(0.f), wa = both(0.f);
                float v[8];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float2 e = fma2(dp, both(cs[s]), g[0][s]);
                    const float2 db = mul2(e, u), dc = mul2(dp, hs[i + 1][s]);
                    v[s] = db.x + db.y;
                    v[4 + s] = dc.x + dc.y;
                    du = fma2(e, both(bs[s]), du);
                    g[0][s] = mul2(al[i][s], e);
                    const float2 ww = mul2(g[0][s], hs[i][s]);
                    wa = fma2(ww, A2[0][s], wa);
                    dA[0][s] = fma2(ww, dt, dA[0][s]);
                }
                // over the warp's channels: value number at.. of dB (four states), dC (four states)
                const int at = spread_sum<8, Q, 32>(v);
                constexpr int kLeft = 32 / Q >= 8 ? 1 : 8 * Q / 32;
                if (cg < 8) {
#pragma unroll
                    for (int j = 0; j < kLeft; ++j) sm.dbc[w][r][(at + j) / 4 * kSP + s0 + (at + j) % 4] = v[j];
                }
                // over the channel's states; every lane has read its u before it takes part
                float t[4] = {du.x, du.y, wa.x, wa.y};
                const int to = spread_sum<4, 1, Q>(t);
                if (Q <= 4 || q < 4) {
#pragma unroll
                    for (int j = 0; j < (Q >= 4 ? 1 : 4 / Q); ++j) {
                        if (to + j < 2) sm.u[r][cl + to + j] = t[j];
                        else sm.r[r][cl + to + j - 2] = t[j];
                    }
                }
            }
        }
        __syncthreads();
        for (int r = r4; r < n; r += kRows) {
            const int64_t tok = blk.start + r;
            const float4 x4 = load4<X>(a.x, tok * a.x_st + tile.ch + c4, cn, a.vec), raw4 = raw_steps<X>(a, tok, tile.ch + c4, cn, bias);
            const float4 dt4 = *reinterpret_cast<const float4*>(&sm.dt[r][c4]), du4 = *reinterpret_cast<const float4*>(&sm.u[r][c4]);
            const float4 dp4 = *reinterpret_cast<const float4*>(&sm.dp[r][c4]), wa4 = *reinterpret_cast<const float4*>(&sm.r[r][c4]);
            const float x[4] = {x4.x, x4.y, x4.z, x4.w}, raw[4] = {raw4.x, raw4.y, raw4.z, raw4.w}, dt[4] = {dt4.x, dt4.y, dt4.z, dt4.w};
            const float du[4] = {du4.x, du4.y, du4.z, du4.w}, dp[4] = {dp4.x, dp4.y, dp4.z, dp4.w}, wa[4] = {wa4.x, wa4.y, wa4.z, wa4.w};
            float dx[4], dd[4];
            constexpr float kLn2 = 0.6931471805599453f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dx[i] = fmaf(du[i], dt[i], dp[i] * skip[i]);
                dd[i] = fmaf(du[i], x[i], wa[i] * kLn2);
                if (a.softplus) dd[i] *= sigmoidf(raw[i]);
                d_skip[i] = fmaf(dp[i], x[i], d_skip[i]);
                d_bias[i] += dd[i];
            }
            store4<X>(a.dx, tok * a.dx_st + tile.ch + c4, cn, a.vec, make_float4(dx[0], dx[1], dx[2], dx[3]));
            store4<X>(a.ddt, tok * a.ddt_st + tile.ch + c4, cn, a.vec, make_float4(dd[0], dd[1], dd[2], dd[3]));
        }
        for (int i = tid; i < n * 2 * kSP; i += kThreads) {
            const int r = i / (2 * kSP), j = i % (2 * kSP), s = j % kSP;
            if (s >= a.S) continue;
            float t = sm.dbc[0][r][j];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) t += sm.dbc[k][r][j];
            const int64_t at = (static_cast<int64_t>(tl - tile.group * a.tiles_pg) * a.T + blk.start + r) * a.G + tile.group;
            a.dbc[(at * 2 + j / kSP) * a.S + s] = t;
        }
    }
    store_thread_states(dA, a.pA, part, a, d0, end, s0, 0);
    // d skip and d bias over the threads that share their channels, in order
    __syncthreads();
    float* red = &sm.dt[0][0];  // [2][kRows][kTile]
    *reinterpret_cast<float4*>(red + r4 * kTile + c4) = make_float4(d_skip[0], d_skip[1], d_skip[2], d_skip[3]);
    *reinterpret_cast<float4*>(red + (kRows + r4) * kTile + c4) = make_float4(d_bias[0], d_bias[1], d_bias[2], d_bias[3]);
    __syncthreads();
    for (int i = tid; i < 2 * kTile; i += kThreads) {
        const int which = i / kTile, c = i % kTile;
        if (c >= tile.n) continue;
        float t = 0.f;
        for (int r = 0; r < kRows; ++r) t += red[(which * kRows + r) * kTile + c];
        a.pch[(static_cast<int64_t>(part) * 2 + which) * a.D + tile.ch + c] = t;
    }
}

// ---------------------------------------------------------------- sums over tiles and parts
template <typename X>
__global__ void __launch_bounds__(256) ssm_sum_bc_kernel(const Args a) {
    const int64_t e = blockIdx.x * 256ll + threadIdx.x, n = a.T * a.G * 2 * a.S;
    if (e >= n) return;
    const float t = strided_sum<8>(a.dbc + e, n, 0, a.tiles_pg, 1);
    const int64_t row = e / (2 * a.S), j = e - row * 2 * a.S;
    X* to = static_cast<X*>(j < a.S ? a.db : a.dc);
    to[row * a.S + (j < a.S ? j : j - a.S)] = from_f<X>(t);
}
__global__ void __launch_bounds__(256) ssm_sum_parts_kernel(const Args a) {
    const int64_t e = blockIdx.x * 256ll + threadIdx.x, DS = static_cast<int64_t>(a.D) * a.S;
    if (e < DS) {
        a.dA[e] = strided_sum<8>(a.pA + e, DS, 0, a.parts, 1);
    } else if (e < DS + 2 * a.D) {
        const int64_t c = e - DS;
        float* to = c < a.D ? a.dskip : a.dbias;
        if (to) to[c < a.D ? c : c - a.D] = strided_sum<8>(a.pch + c, 2 * a.D, 0, a.parts, 1);
    }
}

struct Back {
    template <typename X, int Q>
    static la_status run(Args& a, cudaStream_t s) {
        if (a.N > 0) {
            const int64_t slots = slots_for(a.T, a.N, kShift);
            if (a.T > 0) {
                Args c = a;
                constexpr int kW = 128 / Q;
                c.tiles_pg = (a.Dg + kW - 1) / kW;
                ssm_chunk_gradient_kernel<X, Q><<<slot_grid(c.tiles_pg * a.G, slots), 32, 0, s>>>(c);
            }
            const unsigned bx = static_cast<unsigned>((static_cast<int64_t>(a.D) * a.S + 127) / 128);
            ssm_join_back_kernel<<<slot_grid(static_cast<int>(bx), a.N), 128, 0, s>>>(a);
        }
        constexpr int kTile = Work<Q>::kTile;
        a.tiles_pg = (a.Dg + kTile - 1) / kTile;
        constexpr int kSmem = sizeof(Work<Q>);
        static const cudaError_t opted =
            cudaFuncSetAttribute(ssm_chunk_kernel<X, Q>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (opted != cudaSuccess) return LA_ERR_CUDA;
        ssm_chunk_kernel<X, Q><<<static_cast<unsigned>(a.parts * a.tiles_pg * a.G), kThreads, kSmem, s>>>(a);
        const int64_t n = a.T * a.G * 2 * a.S;
        if (n > 0) ssm_sum_bc_kernel<X><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a);
        ssm_sum_parts_kernel<<<static_cast<unsigned>((static_cast<int64_t>(a.D) * a.S + 2 * a.D + 255) / 256), 256, 0, s>>>(a);
        return launched();
    }
};

}  // namespace

int bwd_width(int S) { return 64 * kWarps / lanes_for(S); }

// How many CTAs share a tile's chunks: enough to fill the GPU three to an SM, none without a chunk.
int bwd_parts(int64_t T, int32_t N, int D, int S, int G) {
    const int width = bwd_width(S);
    const int64_t tiles = static_cast<int64_t>((D / G + width - 1) / width) * G;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(slots_for(T, N, kShift), (3 * kSms + tiles - 1) / tiles)));
}

la_status run_bwd(Args a, int32_t dtype, cudaStream_t s) { return by_shape<Back>(dtype, a.S, a, s); }

}  // namespace ssm
}  // namespace la
