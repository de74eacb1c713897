// glr_bwd.cu -- the backward scan of the gated linear recurrence (glr.cuh has the method).
#include "glr.cuh"

namespace la {
namespace glr {
namespace {

// Warps of a CTA, and CTAs of an SM (as many as the staged rows leave room for).  Short spans: the states before
// each of its tokens stay in registers, or nearly (8 x 8192 x 4096 bf16: 5 % less time with 4 CTAs of 64 registers a
// thread than with 3 of 80).
constexpr int kWarps = 8;
template <typename X, typename G>
constexpr int ctas() { return sizeof(X) == 4 ? 2 : sizeof(G) == 4 ? 3 : 4; }

// 8 x 8192 tokens x 4096 channels, bf16 with logits of a complement gate: 500 us, 5.4 TB/s (80 % of the measured copy
// rate), between its bytes (5 rows) and its issue slots (62 %: the gate evaluated three times).
template <typename X, typename G, int kMode, bool kCompl>
__global__ void __launch_bounds__(32 * kWarps, (ctas<X, G>())) glr_bwd_kernel(const Args a, const __grid_constant__ Maps maps) {
    constexpr int kSpan = span<kWarps>(), kWarpRows = 2 * kSpan;
    extern __shared__ __align__(128) uint8_t stage[];
    __shared__ Shared<kWarps, true> sh;
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
        uint2 seen = make_uint2(kUnset, kUnset);
        if (w == 0 && a.N > 1) seen = peek<true>(a, it);
        if (w == 0 && it.order == 0 && !it.dead && a.dfin)
            load2_any(a.dfin, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, in.x, in.y);
        if (w == 1 && it.count > 0) load2_any(a.ckpt, it.slot * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, in.x, in.y);
        __syncwarp();
        if (a.tma && rows > 0) {
            if (!mbar_wait(&sh.bar[w], parity, kWaitNs, true)) raise_status(a.status, LA_ERR_TIMEOUT);
            parity ^= 1;
        }
        // the maps of the thread's span, h -> ca h + cu forwards and c -> ca c + cc backwards
        Four ca = four(1.f), cu = four(0.f), cc = four(0.f);
        with_span<kSpan>(n, [&](auto whole) {
#pragma unroll
            for (int k = 0; k < kSpan; ++k)
                if (whole || k < n) {
                    const Four x = get4(wx + mine + k * kChannels), g = get4(wg + mine + k * kChannels),
                               d = get4(wd + mine + k * kChannels);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Gated t = gate<kMode, kCompl>(a.lb, g.v[i]);
                        cu.v[i] = fma2(t.a, cu.v[i], kCompl ? mul2(t.m, x.v[i]) : x.v[i]);
                        ca.v[i] = mul2(ca.v[i], t.a);
                        cc.v[i] = fma2(ca.v[i], d.v[i], cc.v[i]);
                    }
                }
        });
        const Four oa = other_half(ca), ou = other_half(cu), oc = other_half(cc);
        if (half == 0) {
            put4(&sh.a[w][c4], mul4(ca, oa));
            put4(&sh.u[w][c4], fma4(oa, cu, ou));
            put4(&sh.c[w][c4], fma4(ca, oc, cc));
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
            chain<true>(a, it, map, seen, in, out);
            *reinterpret_cast<float2*>(&sh.in[2 * lane]) = in;
            if (it.last && !it.dead && a.ds0)
                store2_any(a.ds0, it.state * static_cast<int64_t>(a.D), it.d + 2 * lane, a.D, 0, out.x, out.y);
        }
        // while the chain goes on: the state entering the thread's span, and the gradients' map after it
        Four h = get4(&sh.h0[c4]), pa = four(1.f), pc = four(0.f);
        for (int i = 0; i < w; ++i) h = fma4(get4(&sh.a[i][c4]), h, get4(&sh.u[i][c4]));
        if (half == 1) {
            h = fma4(oa, h, ou);
        } else {
            pa = oa;
            pc = oc;
        }
        for (int i = w + 1; i < kWarps; ++i) {
            pc = fma4(pa, get4(&sh.c[i][c4]), pc);
            pa = mul4(pa, get4(&sh.a[i][c4]));
        }
        __syncthreads();
        if (rows > 0) {
            with_span<kSpan>(n, [&](auto whole) {
                constexpr bool kSlope = kMode != LA_GATE_LOG;
                // forwards for the states before each token; backwards evaluates the gate once more, since
                // keeping it too would not fit the registers
                Four prev[kSpan], e = fma4(pa, get4(&sh.in[c4]), pc);
#pragma unroll
                for (int k = 0; k < kSpan; ++k)
                    if (whole || k < n) {
                        const Four x = get4(wx + mine + k * kChannels), g = get4(wg + mine + k * kChannels);
                        prev[k] = h;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const Gated t = gate<kMode, kCompl>(a.lb, g.v[i]);
                            h.v[i] = fma2(t.a, h.v[i], kCompl ? mul2(t.m, x.v[i]) : x.v[i]);
                            if (kCompl) prev[k].v[i] = fma2(x.v[i], both(-1.f), prev[k].v[i]);
                        }
                    }
                asm volatile("" ::: "memory");  // the compiler would keep the gates, in local memory
#pragma unroll
                for (int k = kSpan - 1; k >= 0; --k)
                    if (whole || k < n) {
                        const Four g = get4(wg + mine + k * kChannels), d = get4(wd + mine + k * kChannels);
                        Four dx, dg;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const Gated t = gate<kMode, kCompl>(a.lb, g.v[i]);
                            e.v[i] = add2(e.v[i], d.v[i]);
                            dx.v[i] = kCompl ? mul2(t.m, e.v[i]) : e.v[i];
                            e.v[i] = mul2(e.v[i], t.a);
                            dg.v[i] = mul2(e.v[i], prev[k].v[i]);
                            if (kSlope) dg.v[i] = mul2(dg.v[i], t.slope);
                        }
                        put4(wx + mine + k * kChannels, dx);
                        put4(wg + mine + k * kChannels, dg);
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
la_status by_gate(Args& a, int32_t xd, int32_t gd, cudaStream_t s) {
    constexpr int kRows = 2 * span<kWarps>();
    Maps maps = {};
    a.tma = row_map(&maps.x, a, a.x, a.x_st, xd, kRows) && row_map(&maps.g, a, a.g, a.g_st, gd, kRows) &&
            row_map(&maps.dh, a, a.dh, a.dh_st, xd, kRows) && row_map(&maps.out, a, a.dx, a.dx_st, xd, kRows) &&
            row_map(&maps.dg, a, a.dg, a.dg_st, gd, kRows);
    la_status st = LA_ERR_INVALID_ARG;
    with_gate(a.mode, a.compl_in, [&](auto gt) {
        st = launch_scan<glr_bwd_kernel<X, G, decltype(gt)::mode, decltype(gt)::complement>>(32 * kWarps, stage_bytes<X, G, 2>(), a, maps, s);
    });
    return st;
}

}  // namespace

la_status run_bwd(Args& a, int32_t xd, int32_t gd, cudaStream_t s) {
    if (xd == LA_DTYPE_BF16) return gd == LA_DTYPE_BF16 ? by_gate<bf16, bf16>(a, xd, gd, s) : by_gate<bf16, float>(a, xd, gd, s);
    return gd == LA_DTYPE_BF16 ? by_gate<float, bf16>(a, xd, gd, s) : by_gate<float, float>(a, xd, gd, s);
}

}  // namespace glr
}  // namespace la
