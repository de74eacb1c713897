// glr_fwd.cu -- the forward scan of the gated linear recurrence (glr.cuh has the method).
#include "glr.cuh"

namespace la {
namespace glr {
namespace {

// Warps of a CTA and CTAs of an SM (as many as the staged rows leave room for).  With 16-bit inputs longer spans leave
// less arithmetic between them (8 x 8192 x 4096, fp32 decays: 4 % less time with 4 warps than with 8; bf16 gates 10 %);
// fp32 rows leave room for three CTAs only, which need the warps (three sequences of 4096 x 2048: 36 and 26 us).
// The unrolling is short because the code is long: 8 tokens at a time cost one long sequence 9 % in instruction misses.
template <typename X, typename G>
constexpr int warps() { return sizeof(X) + sizeof(G) <= 6 ? 4 : 8; }
template <typename X, typename G>
constexpr int ctas() { return sizeof(X) + sizeof(G) == 4 ? 6 : sizeof(X) + sizeof(G) == 6 ? 4 : 3; }

// 8 x 8192 tokens x 4096 channels: bf16 with fp32 decays 340 us, 6.3 TB/s (94 % of the measured copy rate), bound by
// its bytes; with bf16 logits of a complement gate 298 us, 5.4 TB/s, where the gate evaluated twice (17 of 29
// instructions an element) takes over half of the issue slots.  One sequence of 131072 x 1000: 198 us, 4.0 TB/s:
// every block waits for the slowest of the 57 blocks of its channels that are in flight before it.
template <typename X, typename G, int kMode, bool kCompl>
__global__ void __launch_bounds__(32 * warps<X, G>(), (ctas<X, G>())) glr_fwd_kernel(const Args a, const __grid_constant__ Maps maps) {
    constexpr int kWarps = warps<X, G>(), kSpan = span<kWarps>(), kWarpRows = 2 * kSpan;
    extern __shared__ __align__(128) uint8_t stage[];
    __shared__ Shared<kWarps, false> sh;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = lane >> 4, c4 = (lane & 15) * 4;
    X* wx = reinterpret_cast<X*>(stage) + w * kWarpRows * kChannels;                       // the warp's rows
    G* wg = reinterpret_cast<G*>(stage + sizeof(X) * kBlock * kChannels) + w * kWarpRows * kChannels;
    X* sx = wx + half * kSpan * kChannels + c4;                                            // the thread's
    G* sg = wg + half * kSpan * kChannels + c4;
    if (lane == 0) mbar_init(&sh.bar[w], 1);
    fence_mbar_init();
    check_boundaries(a);

    // The warp's rows of an item on their way into shared memory.
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
        uint2 seen = make_uint2(kUnset, kUnset);
        if (w == 0 && a.N > 1) seen = peek<false>(a, it);
        if (w == 0 && it.order == 0 && !it.dead && a.s0)
            load2_any(a.s0, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, a.s0_bf16, in.x, in.y);
        __syncwarp();
        if (a.tma && rows > 0) {
            if (!mbar_wait(&sh.bar[w], parity, kWaitNs, true)) raise_status(a.status, LA_ERR_TIMEOUT);
            parity ^= 1;
        }
        // the map of the thread's span
        Four ca = four(1.f), cu = four(0.f);
        with_span<kSpan>(n, [&](auto whole) {
#pragma unroll (decltype(whole)::value ? 4 : 1)
            for (int k = 0; k < kSpan; ++k)
                if (whole || k < n) {
                    const Four x = get4(sx + k * kChannels), g = get4(sg + k * kChannels);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Gated t = gate<kMode, kCompl>(a.lb, g.v[i]);
                        cu.v[i] = fma2(t.a, cu.v[i], kCompl ? mul2(t.m, x.v[i]) : x.v[i]);
                        ca.v[i] = mul2(ca.v[i], t.a);
                    }
                }
        });
        // the other half's: the lower one's map enters the upper one, both make the warp's
        const Four oa = other_half(ca), ou = other_half(cu);
        if (half == 0) {
            put4(&sh.a[w][c4], mul4(ca, oa));
            put4(&sh.u[w][c4], fma4(oa, cu, ou));
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
            chain<false>(a, it, map, seen, in, out);
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
        Four pa = four(1.f), pu = four(0.f);
        for (int i = 0; i < w; ++i) {
            const Four qa = get4(&sh.a[i][c4]);
            pu = fma4(qa, pu, get4(&sh.u[i][c4]));
            pa = mul4(pa, qa);
        }
        if (half == 1) {
            pu = fma4(oa, pu, ou);
            pa = mul4(pa, oa);
        }
        __syncthreads();
        if (a.h && rows > 0) {
            Four h = fma4(pa, get4(&sh.in[c4]), pu);
            with_span<kSpan>(n, [&](auto whole) {
#pragma unroll (decltype(whole)::value ? 4 : 1)
                for (int k = 0; k < kSpan; ++k)
                    if (whole || k < n) {
                        const Four x = get4(sx + k * kChannels), g = get4(sg + k * kChannels);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const Gated t = gate<kMode, kCompl>(a.lb, g.v[i]);
                            h.v[i] = fma2(t.a, h.v[i], kCompl ? mul2(t.m, x.v[i]) : x.v[i]);
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
la_status by_gate(Args& a, int32_t xd, int32_t gd, cudaStream_t s) {
    constexpr int kWarps = warps<X, G>(), kRows = 2 * span<kWarps>();
    Maps maps = {};
    a.tma = row_map(&maps.x, a, a.x, a.x_st, xd, kRows) && row_map(&maps.g, a, a.g, a.g_st, gd, kRows) &&
            (!a.h || row_map(&maps.out, a, a.h, a.h_st, xd, kRows));
    la_status st = LA_ERR_INVALID_ARG;
    with_gate(a.mode, a.compl_in, [&](auto gt) {
        st = launch_scan<glr_fwd_kernel<X, G, decltype(gt)::mode, decltype(gt)::complement>>(32 * kWarps, stage_bytes<X, G, 1>(), a, maps, s);
    });
    return st;
}

}  // namespace

la_status run_fwd(Args& a, int32_t xd, int32_t gd, cudaStream_t s) {
    if (xd == LA_DTYPE_BF16) return gd == LA_DTYPE_BF16 ? by_gate<bf16, bf16>(a, xd, gd, s) : by_gate<bf16, float>(a, xd, gd, s);
    return gd == LA_DTYPE_BF16 ? by_gate<float, bf16>(a, xd, gd, s) : by_gate<float, float>(a, xd, gd, s);
}

}  // namespace glr
}  // namespace la
