// glr_bwd.cu -- the backward scan of the gated linear recurrence (glr.cuh has the method).
#include "glr.cuh"

namespace la {
namespace glr {
namespace {

// CTAs of an SM: as many as the staged rows leave room for.
template <typename X, typename G>
constexpr int bwd_ctas() { return sizeof(X) + sizeof(G) == 8 ? 2 : 3; }

template <typename X, typename G, int kMode, bool kCompl>
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
        with_span(n, [&](auto whole) {
#pragma unroll
            for (int k = 0; k < kSpan; ++k)
                if (whole || k < n) {
                    float x[4], g[4], d[4];
                    get4(wx + mine + k * kChannels, x);
                    get4(wg + mine + k * kChannels, g);
                    get4(wd + mine + k * kChannels, d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float dec, m, slope;
                        gate<kMode, kCompl>(a.lb, g[i], dec, m, slope);
                        cu[i] = fmaf(dec, cu[i], kCompl ? m * x[i] : x[i]);
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
            with_span(n, [&](auto whole) {
                constexpr bool kSlope = kMode != LA_GATE_LOG;
                // forwards for the states before each token; backwards evaluates the gate once more, since
                // keeping it too would not fit the registers
                float prev[kSpan][4], e[4];
                get4(&sh.in[c4], e);
#pragma unroll
                for (int k = 0; k < kSpan; ++k)
                    if (whole || k < n) {
                        float x[4], g[4];
                        get4(wx + mine + k * kChannels, x);
                        get4(wg + mine + k * kChannels, g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float dec, m, slope;
                            gate<kMode, kCompl>(a.lb, g[i], dec, m, slope);
                            prev[k][i] = h[i];
                            h[i] = fmaf(dec, h[i], kCompl ? m * x[i] : x[i]);
                        }
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = fmaf(pa[i], e[i], pc[i]);
                asm volatile("" ::: "memory");  // the compiler would keep the gates, in local memory
#pragma unroll
                for (int k = kSpan - 1; k >= 0; --k)
                    if (whole || k < n) {
                        float x[4], g[4], d[4];
                        if (kCompl) get4(wx + mine + k * kChannels, x);
                        get4(wg + mine + k * kChannels, g);
                        get4(wd + mine + k * kChannels, d);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float dec, m, slope;
                            gate<kMode, kCompl>(a.lb, g[i], dec, m, slope);
                            e[i] += d[i];
                            d[i] = kCompl ? m * e[i] : e[i];
                            e[i] *= dec;
                            g[i] = e[i] * (kCompl ? prev[k][i] - x[i] : prev[k][i]);
                            if (kSlope) g[i] *= slope;
                        }
                        put4(wx + mine + k * kChannels, d);
                        put4(wg + mine + k * kChannels, g);
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
la_status by_gate(Args& a, Maps& maps, cudaStream_t s) {
    la_status st = LA_ERR_INVALID_ARG;
    with_gate(a.mode, a.compl_in, [&](auto gt) {
        st = launch_scan<glr_bwd_kernel<X, G, decltype(gt)::mode, decltype(gt)::complement>>(stage_bytes<X, G, 2>(), a, maps, s);
    });
    return st;
}

}  // namespace

la_status run_bwd(Args& a, Maps& maps, int32_t xd, int32_t gd, cudaStream_t s) {
    if (xd == LA_DTYPE_BF16) return gd == LA_DTYPE_BF16 ? by_gate<bf16, bf16>(a, maps, s) : by_gate<bf16, float>(a, maps, s);
    return gd == LA_DTYPE_BF16 ? by_gate<float, bf16>(a, maps, s) : by_gate<float, float>(a, maps, s);
}

}  // namespace glr
}  // namespace la
