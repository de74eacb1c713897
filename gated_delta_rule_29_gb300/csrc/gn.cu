// gn.cu -- group norm of every head's channels of every token, with an activation or a gate
// (gn_fwd, gn_bwd).
//
// For one row x[0..V) of a (token, head), with mu = mean(x) (centred) or 0:
//
//   r = 1 / sqrt(mean((x - mu)^2) + eps),  n = (x - mu) r,  p = n w + b,
//   y = act(p)  or  y = p act(z);
//   dp = dy act'(p)  or  dy act(z),   dz = dy p act'(z),   dw = sum dp n,   db = sum dp,
//   dn = dp w,   dx = r (dn - [centred] mean(dn) - n mean(dn n)).
//
// A row is held in the registers of the lanes that share it (a power of two of lanes up to a warp,
// or a whole CTA for long rows), so every operand is read once and every result written once;
// the mean and the variance are two passes over those registers.  The backward recomputes the
// statistics (they are free beside the row's bytes) and each group of lanes keeps to one head, so
// that its weight-gradient sums stay in registers over all its rows; the partial sums of all
// groups are added by a second kernel in a fixed order.
#include <algorithm>

#include "mixer.cuh"

namespace {

using namespace la::mixer;

constexpr int kThreads = 256;
constexpr int kMaxV = 8192;

struct Args {
    const void *x, *z, *w, *b, *dy;
    int64_t x_st, x_sh, z_st, z_sh, dy_st, dy_sh, y_st, y_sh, dz_st, dz_sh;
    int64_t rows, units;  // rows T H; groups of lanes that take part (a multiple of H in the backward)
    int H, V, per_head, center, act, w_bf16;
    int lanes;            // lanes that share a row: 1..32 or kThreads
    float eps;
    void *y, *dz;         // y: the result, or dx in the backward
    float *pw, *pb;       // partial sums [units][V]
};

// Sum over the `lanes` lanes that share a row; kBlock: over the CTA (red has one float per warp).
template <bool kBlock>
__device__ __forceinline__ float row_sum(float v, int lanes, float* red) {
    const int l = kBlock ? 32 : lanes;
    for (int off = l >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (kBlock) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) v += red[i];
    }
    return v;
}

// Element k of a lane is channel lane + k * lanes.
template <typename X, int NE, bool kBlock>
__device__ __forceinline__ void load_row(float (&v)[NE], const void* base, int64_t at, int lane, int lanes, int V) {
#pragma unroll
    for (int k = 0; k < NE; ++k) {
        const int c = lane + k * lanes;
        v[k] = c < V ? to_f(static_cast<const X*>(base)[at + c]) : 0.f;
    }
}

// x becomes n; returns r.
template <int NE, bool kBlock>
__device__ __forceinline__ float normalise(float (&x)[NE], const Args& a, int lane, float* red) {
    float s = 0.f;
    if (a.center) {
#pragma unroll
        for (int k = 0; k < NE; ++k) s += x[k];
        const float mu = row_sum<kBlock>(s, a.lanes, red) / a.V;
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (lane + k * a.lanes < a.V) x[k] -= mu;
        s = 0.f;
    }
#pragma unroll
    for (int k = 0; k < NE; ++k) s = fmaf(x[k], x[k], s);
    const float r = 1.f / sqrtf(row_sum<kBlock>(s, a.lanes, red) / a.V + a.eps);
#pragma unroll
    for (int k = 0; k < NE; ++k) x[k] *= r;
    return r;
}

template <typename X, int NE, bool kBlock>
__global__ void __launch_bounds__(kThreads) gn_fwd_kernel(const Args a) {
    __shared__ float red[kThreads / 32];
    const int lane = threadIdx.x % a.lanes;
    const int64_t unit = blockIdx.x * static_cast<int64_t>(kThreads / a.lanes) + threadIdx.x / a.lanes;
    // every lane of a warp runs the same number of rounds: the shuffles need them all
    const int64_t rounds = (a.rows + a.units - 1) / a.units;
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t row = min(unit + k * a.units, a.rows - 1);
        const bool live = unit + k * a.units < a.rows;
        const int64_t t = row / a.H;
        const int h = static_cast<int>(row % a.H);
        float x[NE];
        load_row<X, NE, kBlock>(x, a.x, t * a.x_st + h * a.x_sh, lane, a.lanes, a.V);
        normalise<NE, kBlock>(x, a, lane, red);
        const int64_t wo = a.per_head ? static_cast<int64_t>(h) * a.V : 0;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int c = lane + e * a.lanes;
            if (c >= a.V || !live) continue;
            float p = x[e] * load_any(a.w, wo + c, a.w_bf16);
            if (a.b) p += load_any(a.b, wo + c, a.w_bf16);
            const float y = a.z ? p * act_fwd(a.act, to_f(static_cast<const X*>(a.z)[t * a.z_st + h * a.z_sh + c]))
                                : act_fwd(a.act, p);
            static_cast<X*>(a.y)[t * a.y_st + h * a.y_sh + c] = from_f<X>(y);
        }
    }
}

template <typename X, int NE, bool kBlock>
__global__ void __launch_bounds__(kThreads) gn_bwd_kernel(const Args a) {
    __shared__ float red[kThreads / 32];
    const int lane = threadIdx.x % a.lanes;
    const int64_t unit = blockIdx.x * static_cast<int64_t>(kThreads / a.lanes) + threadIdx.x / a.lanes;
    const int64_t rounds = (a.rows + a.units - 1) / a.units;
    const int64_t wo = a.per_head ? (unit % a.H) * a.V : 0;
    float w[NE], b[NE], dw[NE], db[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int c = lane + e * a.lanes;
        dw[e] = db[e] = 0.f;
        w[e] = c < a.V ? load_any(a.w, wo + c, a.w_bf16) : 0.f;
        b[e] = c < a.V && a.b ? load_any(a.b, wo + c, a.w_bf16) : 0.f;
    }
    for (int64_t k = 0; k < rounds; ++k) {
        const bool live = unit < a.units && unit + k * a.units < a.rows;
        const int64_t row = live ? unit + k * a.units : 0;
        const int64_t t = row / a.H;
        const int h = static_cast<int>(row % a.H);
        float n[NE], g[NE];
        load_row<X, NE, kBlock>(n, a.x, t * a.x_st + h * a.x_sh, lane, a.lanes, a.V);
        load_row<X, NE, kBlock>(g, a.dy, t * a.dy_st + h * a.dy_sh, lane, a.lanes, a.V);
        const float r = normalise<NE, kBlock>(n, a, lane, red);
        float sg = 0.f, sgn = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int c = lane + e * a.lanes;
            if (c >= a.V) continue;
            const float p = fmaf(n[e], w[e], b[e]);
            float d;
            if (a.z) {
                const float f = act_grad(a.act, to_f(static_cast<const X*>(a.z)[t * a.z_st + h * a.z_sh + c]), d);
                if (live) static_cast<X*>(a.dz)[t * a.dz_st + h * a.dz_sh + c] = from_f<X>(g[e] * p * d);
                g[e] *= f;
            } else {
                act_grad(a.act, p, d);
                g[e] *= d;
            }
            if (live) {
                dw[e] = fmaf(g[e], n[e], dw[e]);
                db[e] += g[e];
            }
            g[e] *= w[e];
            sg += g[e];
            sgn = fmaf(g[e], n[e], sgn);
        }
        const float mg = a.center ? row_sum<kBlock>(sg, a.lanes, red) / a.V : 0.f;
        const float mgn = row_sum<kBlock>(sgn, a.lanes, red) / a.V;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int c = lane + e * a.lanes;
            if (c < a.V && live)
                static_cast<X*>(a.y)[t * a.y_st + h * a.y_sh + c] = from_f<X>(r * (g[e] - mg - n[e] * mgn));
        }
    }
    if (unit >= a.units) return;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int c = lane + e * a.lanes;
        if (c >= a.V) continue;
        a.pw[unit * a.V + c] = dw[e];
        if (a.pb) a.pb[unit * a.V + c] = db[e];
    }
}

// out[c] = sum of the partial sums of column c: rows c / V, + heads, + 2 heads, ... (per head), or
// all rows (shared).  A CTA takes 32 columns; its warps take every eighth row, in order.
__global__ void __launch_bounds__(256) gn_sum_kernel(const float* pw, const float* pb, int64_t units, int V, int heads,
                                                     void* dw, void* db, int w_bf16) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32ll + lane;
    const float* p = blockIdx.y ? pb : pw;
    float s = 0.f;
    if (c < static_cast<int64_t>(V) * heads)
        for (int64_t u = c / V + static_cast<int64_t>(w) * heads; u < units; u += 8ll * heads) s += p[u * V + c % V];
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < static_cast<int64_t>(V) * heads) {
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        store_any(blockIdx.y ? db : dw, c, w_bf16, s);
    }
}

// Lanes that share a row of n elements when each holds at most `most`.
int row_lanes(int n, int most) {
    int l = 1;
    while (l < 32 && l * 4 < n) l *= 2;
    return l * most >= n ? l : kThreads;
}

constexpr int kPerLane = 32;

int64_t bwd_units(int64_t rows, int H, int V) {
    const int per_cta = kThreads / row_lanes(V, kPerLane);
    int64_t u = std::max<int64_t>(1, std::min<int64_t>(rows / 16, 152 * 8 * static_cast<int64_t>(per_cta)));
    return (u + H - 1) / H * H;
}

template <typename X, int NE, bool kBlock>
la_status launch(Args& a, bool bwd, cudaStream_t s) {
    const int64_t per_cta = kThreads / a.lanes;
    if (bwd) {
        const int64_t grid = (a.units + per_cta - 1) / per_cta;
        gn_bwd_kernel<X, NE, kBlock><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
    } else {
        const int64_t grid = std::min<int64_t>((a.rows + per_cta - 1) / per_cta, 152 * 64);
        a.units = grid * per_cta;
        gn_fwd_kernel<X, NE, kBlock><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
    }
    return launched();
}

template <typename X>
la_status dispatch(Args& a, bool bwd, cudaStream_t s) {
    a.lanes = row_lanes(a.V, kPerLane);
    if (a.lanes == kThreads) return launch<X, kPerLane, true>(a, bwd, s);
    if (a.lanes * 4 >= a.V) return launch<X, 4, false>(a, bwd, s);
    return launch<X, kPerLane, false>(a, bwd, s);
}

bool good_thd(const void* p, int64_t st, int64_t sh, int64_t T, int H, int V, int32_t dtype, bool out) {
    if (T == 0) return true;
    if (!p || !aligned_to(p, dtype_size(dtype)) || st < 0 || sh < 0) return false;
    if (!out) return true;
    if (H > 1 && sh < V) return false;
    return T == 1 || st >= V;
}

la_status check(int64_t T, int H, int V, int32_t xd, int32_t wd, int32_t act, float eps, const void* w, const void* b) {
    if (T < 0 || H <= 0 || V <= 0) return LA_ERR_INVALID_ARG;
    if (!known_dtype(xd) || !known_dtype(wd)) return LA_ERR_UNSUPPORTED;
    if (act < LA_ACT_NONE || act > LA_ACT_SIGMOID) return LA_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    if (V > kMaxV || T >= (int64_t(1) << 40) / H) return LA_ERR_UNSUPPORTED;
    if (!w || !aligned_to(w, dtype_size(wd)) || !good_optional(b, wd)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

}  // namespace

extern "C" {

size_t la_gn_bwd_workspace_bytes(int64_t T, int32_t H, int32_t V, int32_t per_head) {
    if (T < 0 || H <= 0 || V <= 0 || V > kMaxV) return 0;
    return static_cast<size_t>(bwd_units(T * H, H, V)) * V * 2 * 4 + 256;
}

la_status gn_fwd(const la_gn_fwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check(p->T, p->H, p->V, p->x_dtype, p->weight_dtype, p->activation, p->eps, p->weight, p->bias);
    if (st != LA_OK) return st;
    if (!good_thd(p->x, p->x_stride_t, p->x_stride_h, p->T, p->H, p->V, p->x_dtype, false) ||
        (p->z && !good_thd(p->z, p->z_stride_t, p->z_stride_h, p->T, p->H, p->V, p->x_dtype, false)) ||
        !good_thd(p->y, p->y_stride_t, p->y_stride_h, p->T, p->H, p->V, p->x_dtype, true))
        return LA_ERR_INVALID_ARG;
    if (p->T == 0) return LA_OK;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.x_sh = p->x_stride_h;
    a.z = p->z; a.z_st = p->z_stride_t; a.z_sh = p->z_stride_h;
    a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.rows = p->T * p->H; a.H = p->H; a.V = p->V;
    a.per_head = p->per_head != 0; a.center = p->center != 0; a.act = p->activation; a.eps = p->eps;
    a.y = p->y; a.y_st = p->y_stride_t; a.y_sh = p->y_stride_h;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return p->x_dtype == LA_DTYPE_BF16 ? dispatch<bf16>(a, false, s) : dispatch<float>(a, false, s);
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
    a.rows = p->T * p->H; a.H = p->H; a.V = p->V;
    a.per_head = p->per_head != 0; a.center = p->center != 0; a.act = p->activation; a.eps = p->eps;
    a.y = p->dx; a.y_st = p->dx_stride_t; a.y_sh = p->dx_stride_h;
    a.dz = p->dz; a.dz_st = p->dz_stride_t; a.dz_sh = p->dz_stride_h;
    a.units = bwd_units(a.rows, a.H, a.V);
    a.pw = static_cast<float*>(p->workspace);
    a.pb = p->bias ? a.pw + a.units * a.V : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t units = a.units;
    if (p->T > 0) {
        st = p->x_dtype == LA_DTYPE_BF16 ? dispatch<bf16>(a, true, s) : dispatch<float>(a, true, s);
        if (st != LA_OK) return st;
    } else {
        units = 0;  // no rows: the sums are zero
    }
    const int heads = a.per_head ? a.H : 1;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.V) * heads + 31) / 32), a.pb ? 2 : 1);
    gn_sum_kernel<<<grid, 256, 0, s>>>(a.pw, a.pb, units, a.V, heads, p->d_weight, p->d_bias, a.w_bf16);
    return launched();
}

}  // extern "C"
