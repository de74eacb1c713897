// gn_bwd.cu -- the group norm's backward (gn.cuh has the method).
#include "gn.cuh"

namespace la {
namespace gn {
namespace {

template <typename X, int kVec, int NV, bool kBias>
constexpr int resident() { return ctas(NV * kVec, 1, kBias || sizeof(X) == 4 || kVec < 4 ? 2 : 3); }
constexpr int kMostResident = 3;

// Bound by its bytes where there are many (5 rows with a gate): 65536 x 32 x 128 bf16 in 430 us, 6.2 TB/s (93 % of
// the measured copy rate); the paired arithmetic took 50 us off.  Small batches are bound by the rounds of a
// group, each a load, two to four reductions over its lanes and a store: 4099 x 10 x 100, 16 us of a 4 us floor.
template <typename X, int kVec, int NV, bool kBlock, bool kBias>
__global__ void __launch_bounds__(kThreads, (resident<X, kVec, NV, kBias>())) gn_bwd_kernel(const Args a) {
    extern __shared__ float sums[];  // [groups][V]: one weight gradient's sums at a time
    __shared__ float red[kThreads / 32];
    const int lane = threadIdx.x % a.lanes;
    const Walk r = walk(a);
    const int64_t rounds = (a.T + r.step - 1) / r.step;
    const float inv_v = 1.f / a.V;
    constexpr int kPairs = NV * kVec / 2;
    float2 w[kPairs], b[kPairs], dw[kPairs], db[kPairs];  // b and db: unused without a bias
    Packed<X, kVec> raw[NV], z[NV], dy[NV], next[NV], next_z[NV], next_dy[NV];
    auto load = [&](Packed<X, kVec> (&x)[NV], Packed<X, kVec> (&g)[NV], Packed<X, kVec> (&d)[NV], int64_t t) {
        load_row<X, kVec, NV>(x, a.x, t * a.x_st + r.h * a.x_sh, t < a.T, lane, a);
        load_row<X, kVec, NV>(d, a.dy, t * a.dy_st + r.h * a.dy_sh, t < a.T, lane, a);
        if (a.z) load_row<X, kVec, NV>(g, a.z, t * a.z_st + r.h * a.z_sh, t < a.T, lane, a);
    };
    constexpr bool kAhead = NV * kVec <= 8 && kVec * sizeof(X) >= 8;
    int64_t t = r.t0;
    if (kAhead) load(next, next_z, next_dy, t);
    load_weights<kVec, NV>(w, a.w, r.h, lane, a);
    if (kBias) load_weights<kVec, NV>(b, a.b, r.h, lane, a);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) dw[j] = db[j] = both(0.f);
    for (int64_t round = 0; round < rounds; ++round, t += r.step) {
        const bool live = t < a.T;
        if (kAhead) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                raw[k] = next[k];
                z[k] = next_z[k];
                dy[k] = next_dy[k];
            }
            load(next, next_z, next_dy, t + r.step);
        } else {
            load(raw, z, dy, t);
        }
        float2 n[kPairs], g[kPairs], sg = both(0.f), sgn = both(0.f);
        const float rs = normalise<X, kVec, NV, kBlock>(raw, n, a, inv_v, lane, red);
        X* to_dz = static_cast<X*>(a.dz) + t * a.dz_st + r.h * a.dz_sh;
        with_act(a, [&](auto act, auto gated) {
            float2 dz[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 p = kBias ? fma2(n[j], w[j], b[j]) : mul2(n[j], w[j]);
                const float2 v = pair_of<X, kVec, NV>(dy, j);  // 0 beyond V and where not live, and so is all that follows from it
                float2 d;
                if (gated) {
                    const float2 f = act_grad2<act>(pair_of<X, kVec, NV>(z, j), d);
                    dz[j] = mul2(mul2(v, p), d);
                    g[j] = mul2(v, f);
                } else {
                    act_grad2<act>(p, d);
                    g[j] = mul2(v, d);
                }
            }
            if (gated && live) store_row<X, kVec, NV>(to_dz, dz, lane, a);
        });
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            dw[j] = fma2(g[j], n[j], dw[j]);
            if (kBias) db[j] = add2(db[j], g[j]);
            g[j] = mul2(g[j], w[j]);
            sg = add2(sg, g[j]);
            sgn = fma2(g[j], n[j], sgn);
        }
        const float mg = a.center ? row_sum<kBlock>(sg.x + sg.y, a.lanes, red) * inv_v : 0.f;
        const float mgn = row_sum<kBlock>(sgn.x + sgn.y, a.lanes, red) * inv_v;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) g[j] = mul2(both(rs), fma2(n[j], both(-mgn), add2(g[j], both(-mg))));
        store_row<X, kVec, NV>(static_cast<X*>(a.y) + t * a.y_st + r.h * a.y_sh, g, lane, a);
    }
    // the CTA's sums, group by group
    const int groups = kThreads / a.lanes, u = threadIdx.x / a.lanes;
#pragma unroll
    for (int which = 0; which < (kBias ? 2 : 1); ++which) {
        float* out = which ? a.pb : a.pw;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < NV * kVec; ++e) {
            const int c = (lane + e / kVec * a.lanes) * kVec + e % kVec;
            const float2 v = which ? db[e / 2] : dw[e / 2];
            if (c < a.V) sums[u * a.V + c] = e % 2 ? v.y : v.x;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.V; c += kThreads) {
            float s = 0.f;
            for (int q = 0; q < groups; ++q) s += sums[q * a.V + c];
            out[static_cast<int64_t>(blockIdx.x) * a.V + c] = s;
        }
    }
}

// 456 rows of 128 in 4.6 us: a launch and two round trips, not bytes.
// out[c] = the sum over the CTAs' partial sums of column c: rows c / V, + heads, + 2 heads, ... (per
// head), or all rows (shared).  A CTA takes 32 columns; its 32 warps take every 32nd row, in order.
__global__ void __launch_bounds__(1024) gn_sum_kernel(const float* pw, const float* pb, int64_t rows, int V, int heads,
                                                      void* dw, void* db, int w_bf16) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32ll + lane;
    const float* p = blockIdx.y ? pb : pw;
    float s = 0.f;
    if (c < static_cast<int64_t>(V) * heads) {
        const int64_t step = 32ll * heads;
        s = strided_sum<16>(p + c % V, V, c / V + static_cast<int64_t>(w) * heads, rows, step);
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < static_cast<int64_t>(V) * heads) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += part[i][lane];
        store_any(blockIdx.y ? db : dw, c, w_bf16, s);
    }
}

// CTAs of the backward, per_sm an SM at most: at least kMinRows rows for a group of lanes, and a multiple of the heads where
// each CTA keeps to one.  The lanes of a row do not depend on its alignment, so the most that any form of a shape takes
// follows from the shape, and with it the workspace's size.
constexpr int kMinRows = 8;
int64_t bwd_ctas(int64_t T, int H, int V, int per_head, int per_sm) {
    const int64_t rows = T * H, groups = kThreads / shape(V, 1).lanes;
    const int64_t n = std::min<int64_t>(std::max<int64_t>(1, rows / kMinRows / groups), static_cast<int64_t>(kSms) * per_sm);
    return per_head ? std::max<int64_t>(H, n / H * H) : std::max(n, (H + groups - 1) / groups);
}

struct Launch {
    template <typename X, int kVec, int NV, bool kBlock>
    static la_status run(Args& a, cudaStream_t s) {
        const int groups = kThreads / a.lanes;
        const size_t smem = static_cast<size_t>(groups) * a.V * sizeof(float);
        a.ctas = bwd_ctas(a.T, a.H, a.V, a.per_head, a.b ? resident<X, kVec, NV, true>() : resident<X, kVec, NV, false>());
        const unsigned grid = static_cast<unsigned>(a.ctas);
        if (a.b) gn_bwd_kernel<X, kVec, NV, kBlock, true><<<grid, kThreads, smem, s>>>(a);
        else gn_bwd_kernel<X, kVec, NV, kBlock, false><<<grid, kThreads, smem, s>>>(a);
        return launched();
    }
};

}  // namespace
}  // namespace gn
}  // namespace la

using namespace la;
using namespace la::mixer;
using namespace la::gn;

extern "C" {

size_t la_gn_bwd_workspace_bytes(int64_t T, int32_t H, int32_t V, int32_t per_head) {
    if (T < 0 || H <= 0 || V <= 0 || V > kMaxV) return 0;
    return (static_cast<size_t>(bwd_ctas(T, H, V, per_head != 0, kMostResident)) * V * 2 * 4 + 255) & ~size_t(255);
}

la_status gn_bwd(const la_gn_bwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check(p->T, p->H, p->V, p->x_dtype, p->weight_dtype, p->activation, p->eps, p->weight, p->bias);
    if (st != LA_OK) return st;
    if (!good_thd(p->x, p->x_stride_t, p->x_stride_h, p->T, p->H, p->V, p->x_dtype, false) ||
        !good_thd(p->dy, p->dy_stride_t, p->dy_stride_h, p->T, p->H, p->V, p->x_dtype, false) ||
        !good_thd(p->dx, p->dx_stride_t, p->dx_stride_h, p->T, p->H, p->V, p->x_dtype, true) ||
        (p->z && (!good_thd(p->z, p->z_stride_t, p->z_stride_h, p->T, p->H, p->V, p->x_dtype, false) ||
                  !good_thd(p->dz, p->dz_stride_t, p->dz_stride_h, p->T, p->H, p->V, p->x_dtype, true))))
        return LA_ERR_INVALID_ARG;
    if (!p->d_weight || !aligned_to(p->d_weight, dtype_size(p->weight_dtype)) || (p->bias && !p->d_bias) ||
        !good_optional(p->d_bias, p->weight_dtype))
        return LA_ERR_INVALID_ARG;
    if ((st = check_workspace(p->workspace, p->workspace_bytes,
                              la_gn_bwd_workspace_bytes(p->T, p->H, p->V, p->per_head))) != LA_OK)
        return st;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.x_sh = p->x_stride_h;
    a.z = p->z; a.z_st = p->z_stride_t; a.z_sh = p->z_stride_h;
    a.dy = p->dy; a.dy_st = p->dy_stride_t; a.dy_sh = p->dy_stride_h;
    a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.T = p->T; a.H = p->H; a.V = p->V;
    a.per_head = p->per_head != 0; a.center = p->center != 0; a.act = p->activation; a.eps = p->eps;
    a.y = p->dx; a.y_st = p->dx_stride_t; a.y_sh = p->dx_stride_h;
    a.dz = p->dz; a.dz_st = p->dz_stride_t; a.dz_sh = p->dz_stride_h;
    a.pw = static_cast<float*>(p->workspace);
    a.pb = p->bias ? a.pw + bwd_ctas(a.T, a.H, a.V, a.per_head, kMostResident) * a.V : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->T > 0) {
        st = p->x_dtype == LA_DTYPE_BF16 ? dispatch<Launch, bf16>(a, s) : dispatch<Launch, float>(a, s);
        if (st != LA_OK) return st;
    }
    const int heads = a.per_head ? a.H : 1;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.V) * heads + 31) / 32), a.pb ? 2 : 1);
    gn_sum_kernel<<<grid, 1024, 0, s>>>(a.pw, a.pb, a.ctas, a.V, heads, p->d_weight, p->d_bias, a.w_bf16);
    return launched();
}

}  // extern "C"
