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
// A row is held in the registers of the lanes that share it (a power of two of lanes up to a warp, or a
// whole CTA for long rows), so every operand is read once and every result written once, 16 bytes a
// lane where the rows' alignment allows; the mean and the variance are two passes over those registers.
// A group of lanes keeps to one head and steps over the tokens, so that the weights stay in registers.
// The backward recomputes the statistics (they are free beside the row's bytes) and keeps the weight
// gradients' sums in registers over all its rows; a CTA adds its groups' sums and a second kernel the
// CTAs', both in a fixed order.
#include <algorithm>
#include <type_traits>

#include "mixer.cuh"

namespace {

using namespace la::mixer;

constexpr int kThreads = 256;
constexpr int kMaxV = 8192;

struct Args {
    const void *x, *z, *w, *b, *dy;
    int64_t x_st, x_sh, z_st, z_sh, dy_st, dy_sh, y_st, y_sh, dz_st, dz_sh;
    int64_t T;
    int H, V, per_head, center, act, w_bf16;
    int lanes;            // lanes that share a row: 1..32 or kThreads
    float eps;
    void *y, *dz;         // y: the result, or dx in the backward
    float *pw, *pb;       // partial sums [CTAs][V]
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

// The rows of a group of lanes: head h, tokens t0, t0 + step, ...  With weights of their own every CTA
// keeps to one head (the CTAs' sums are then the heads'); with shared weights neighbouring groups take
// neighbouring rows, and the groups beyond the last multiple of H have none (t0 = T).
struct Walk {
    int h;
    int64_t t0, step;
};
__device__ __forceinline__ Walk walk(const Args& a) {
    Walk r;
    const int per_cta = kThreads / a.lanes, u = threadIdx.x / a.lanes;
    if (a.per_head) {
        r.h = blockIdx.x % a.H;
        r.t0 = static_cast<int64_t>(blockIdx.x / a.H) * per_cta + u;
        r.step = static_cast<int64_t>(gridDim.x / a.H) * per_cta;
    } else {
        const int64_t unit = static_cast<int64_t>(blockIdx.x) * per_cta + u;
        r.step = static_cast<int64_t>(gridDim.x) * per_cta / a.H;
        r.t0 = unit / a.H;
        r.h = static_cast<int>(unit - r.t0 * a.H);
        if (r.t0 >= r.step) r.t0 = a.T;
    }
    return r;
}

// A lane's part of a row: NV vectors of kVec elements, vector k from channel (lane + k * lanes) * kVec on; in fp32 as
// pairs, element e being element e % kVec of vector e / kVec.
template <typename X, int kVec, int NV>
__device__ __forceinline__ void load_row(Packed<X, kVec> (&v)[NV], const void* base, int64_t at, bool live, int lane, const Args& a) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * a.lanes) * kVec;
        if (live && c < a.V) v[k].load(static_cast<const X*>(base) + at + c);
        else v[k].zero();
    }
}
template <typename X, int kVec, int NV>
__device__ __forceinline__ float2 pair_of(const Packed<X, kVec> (&v)[NV], int j) {
    return make_float2(v[2 * j / kVec].get(2 * j % kVec), v[(2 * j + 1) / kVec].get((2 * j + 1) % kVec));
}
template <typename X, int kVec, int NV>
__device__ __forceinline__ void store_row(X* to, const float2 (&v)[NV * kVec / 2], int lane, const Args& a) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * a.lanes) * kVec;
        float y[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = (k * kVec + i) % 2 ? v[(k * kVec + i) / 2].y : v[(k * kVec + i) / 2].x;
        if (c < a.V) store_packed<X, kVec>(to + c, y);
    }
}

// n from a row; returns r.  Places beyond V stay 0.
template <typename X, int kVec, int NV, bool kBlock>
__device__ __forceinline__ float normalise(const Packed<X, kVec> (&raw)[NV], float2 (&x)[NV * kVec / 2], const Args& a, float inv_v, int lane, float* red) {
    constexpr int kPairs = NV * kVec / 2;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) x[j] = pair_of<X, kVec, NV>(raw, j);
    float2 s;
    if (a.center) {
        s = x[0];
#pragma unroll
        for (int j = 1; j < kPairs; ++j) s = add2(s, x[j]);
        const float mu = row_sum<kBlock>(s.x + s.y, a.lanes, red) * inv_v;
        // what is subtracted from each of a pair's elements: the mean, but 0 beyond V
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const int k0 = 2 * j / kVec, k1 = (2 * j + 1) / kVec;
            x[j] = add2(x[j], make_float2((lane + k0 * a.lanes) * kVec < a.V ? -mu : 0.f, (lane + k1 * a.lanes) * kVec < a.V ? -mu : 0.f));
        }
    }
    s = mul2(x[0], x[0]);
#pragma unroll
    for (int j = 1; j < kPairs; ++j) s = fma2(x[j], x[j], s);
    const float v = fmaf(row_sum<kBlock>(s.x + s.y, a.lanes, red), inv_v, a.eps);
    // the reciprocal square root and one step of Newton's method for 1 / r^2 = v (where r^2 v is finite)
    const float r0 = rsqrtf(v), e = fmaf(-v * r0, r0, 1.f), r = fabsf(e) < 0.5f ? fmaf(0.5f * r0, e, r0) : r0;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) x[j] = mul2(x[j], both(r));
    return r;
}

// A parameter's values for a lane's channels.
template <typename W, int kVec, int NV>
__device__ __forceinline__ void load_parameter(float2 (&w)[NV * kVec / 2], const void* p, int64_t at, int lane, const Args& a) {
    float e[NV * kVec];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = (lane + k * a.lanes) * kVec + i;
            e[k * kVec + i] = p && c < a.V ? to_f(static_cast<const W*>(p)[at + c]) : 0.f;
        }
#pragma unroll
    for (int j = 0; j < NV * kVec / 2; ++j) w[j] = make_float2(e[2 * j], e[2 * j + 1]);
}
template <int kVec, int NV>
__device__ __forceinline__ void load_weights(float2 (&w)[NV * kVec / 2], const void* p, int h, int lane, const Args& a) {
    const int64_t at = a.per_head ? static_cast<int64_t>(h) * a.V : 0;
    if (a.w_bf16) load_parameter<bf16, kVec, NV>(w, p, at, lane, a);
    else load_parameter<float, kVec, NV>(w, p, at, lane, a);
}

// Calls f with the activation and whether it is a gate's as constants.
template <typename F>
__device__ __forceinline__ void with_act(const Args& a, F f) {
    typedef std::integral_constant<int, LA_ACT_NONE> None;
    typedef std::integral_constant<int, LA_ACT_SILU> Silu;
    typedef std::integral_constant<int, LA_ACT_SIGMOID> Sigmoid;
    if (a.z) {
        if (a.act == LA_ACT_SILU) f(Silu(), std::true_type());
        else if (a.act == LA_ACT_SIGMOID) f(Sigmoid(), std::true_type());
        else f(None(), std::true_type());
    } else {
        if (a.act == LA_ACT_SILU) f(Silu(), std::false_type());
        else if (a.act == LA_ACT_SIGMOID) f(Sigmoid(), std::false_type());
        else f(None(), std::false_type());
    }
}

// Resident CTAs to compile for: more, with fewer registers each, where a lane holds little.
constexpr int ctas(int elements, int few, int many) { return elements <= 8 ? many : elements <= 16 ? few : 1; }

template <typename X, int kVec, int NV, bool kBlock>
__global__ void __launch_bounds__(kThreads, ctas(NV * kVec, 2, sizeof(X) == 4 ? 3 : 4)) gn_fwd_kernel(const Args a) {
    __shared__ float red[kThreads / 32];
    const int lane = threadIdx.x % a.lanes;
    const Walk r = walk(a);
    const int64_t rounds = (a.T + r.step - 1) / r.step;  // the same for every lane of a warp: the shuffles need them all
    const float inv_v = 1.f / a.V;
    constexpr int kPairs = NV * kVec / 2;
    float2 w[kPairs], b[kPairs];
    load_weights<kVec, NV>(w, a.w, r.h, lane, a);
    load_weights<kVec, NV>(b, a.b, r.h, lane, a);
    Packed<X, kVec> raw[NV], z[NV], next[NV], next_z[NV];
    auto load = [&](Packed<X, kVec> (&x)[NV], Packed<X, kVec> (&g)[NV], int64_t t) {
        load_row<X, kVec, NV>(x, a.x, t * a.x_st + r.h * a.x_sh, t < a.T, lane, a);
        if (a.z) load_row<X, kVec, NV>(g, a.z, t * a.z_st + r.h * a.z_sh, t < a.T, lane, a);
    };
    // short rows: the next one is on its way while this one is worked on
    constexpr bool kAhead = NV * kVec <= 8;
    int64_t t = r.t0;
    if (kAhead) load(next, next_z, t);
    for (int64_t n = 0; n < rounds; ++n, t += r.step) {
        const bool live = t < a.T;
        if (kAhead) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                raw[k] = next[k];
                z[k] = next_z[k];
            }
            load(next, next_z, t + r.step);
        } else {
            load(raw, z, t);
        }
        float2 x[kPairs];
        normalise<X, kVec, NV, kBlock>(raw, x, a, inv_v, lane, red);
        if (!live) continue;
        with_act(a, [&](auto act, auto gated) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 p = fma2(x[j], w[j], b[j]);
                x[j] = gated ? mul2(p, act_fwd2<act>(pair_of<X, kVec, NV>(z, j))) : act_fwd2<act>(p);
            }
        });
        store_row<X, kVec, NV>(static_cast<X*>(a.y) + t * a.y_st + r.h * a.y_sh, x, lane, a);
    }
}

template <typename X, int kVec, int NV, bool kBlock, bool kBias>
__global__ void __launch_bounds__(kThreads, ctas(NV * kVec, 1, kBias || sizeof(X) == 4 ? 2 : 3)) gn_bwd_kernel(const Args a) {
    extern __shared__ float sums[];  // [groups][V]: one weight gradient's sums at a time
    __shared__ float red[kThreads / 32];
    const int lane = threadIdx.x % a.lanes;
    const Walk r = walk(a);
    const int64_t rounds = (a.T + r.step - 1) / r.step;
    const float inv_v = 1.f / a.V;
    constexpr int kPairs = NV * kVec / 2;
    float2 w[kPairs], b[kPairs], dw[kPairs], db[kPairs];  // b and db: unused without a bias
    load_weights<kVec, NV>(w, a.w, r.h, lane, a);
    if (kBias) load_weights<kVec, NV>(b, a.b, r.h, lane, a);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) dw[j] = db[j] = both(0.f);
    Packed<X, kVec> raw[NV], z[NV], dy[NV], next[NV], next_z[NV], next_dy[NV];
    auto load = [&](Packed<X, kVec> (&x)[NV], Packed<X, kVec> (&g)[NV], Packed<X, kVec> (&d)[NV], int64_t t) {
        load_row<X, kVec, NV>(x, a.x, t * a.x_st + r.h * a.x_sh, t < a.T, lane, a);
        load_row<X, kVec, NV>(d, a.dy, t * a.dy_st + r.h * a.dy_sh, t < a.T, lane, a);
        if (a.z) load_row<X, kVec, NV>(g, a.z, t * a.z_st + r.h * a.z_sh, t < a.T, lane, a);
    };
    constexpr bool kAhead = NV * kVec <= 8;
    int64_t t = r.t0;
    if (kAhead) load(next, next_z, next_dy, t);
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
#pragma unroll 8
        for (int64_t u = c / V + static_cast<int64_t>(w) * heads; u < rows; u += step) s += p[u * V + c % V];
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < static_cast<int64_t>(V) * heads) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += part[i][lane];
        store_any(blockIdx.y ? db : dw, c, w_bf16, s);
    }
}

// ---------------------------------------------------------------- shapes
// How a row is spread over lanes: vectors of 16 bytes, of 8 (bf16), or single elements; as few lanes as hold it at 8
// elements each, up to a warp (the fewer lanes, the fewer shuffles a row), then up to kPerLane elements a lane, then
// the whole CTA.
constexpr int kPerLane = 32;

struct Shape {
    int lanes, nv;
};
Shape shape(int V, int vec) {
    const int n = (V + vec - 1) / vec;  // vectors
    Shape s = {1, 1};
    while (s.lanes < 32 && s.lanes * (8 / vec) < n) s.lanes *= 2;
    if (V > 32 * kPerLane) s.lanes = kThreads;
    s.nv = (n + s.lanes - 1) / s.lanes;
    return s;
}

// CTAs of the backward: a few waves' worth, with at least kMinRows rows for a group of lanes, and a
// multiple of the heads where each CTA keeps to one.  The lanes of a row do not depend on its alignment, so the
// workspace's size follows from the shape.
constexpr int kMaxCtas = 152 * 6, kMinRows = 8;
int64_t bwd_ctas(int64_t T, int H, int V, int per_head) {
    const int64_t rows = T * H, most = rows / kMinRows;
    const int64_t groups = kThreads / shape(V, 1).lanes;
    int64_t n = std::max<int64_t>(1, std::min<int64_t>(kMaxCtas, most / groups));
    if (per_head) n = (n + H - 1) / H * H;
    else n = std::max(n, (H + groups - 1) / groups);
    return n;
}

template <typename X, int kVec, int NV, bool kBlock>
la_status launch(const Args& a, bool bwd, cudaStream_t s) {
    const int groups = kThreads / a.lanes;
    if (bwd) {
        const size_t smem = static_cast<size_t>(groups) * a.V * sizeof(float);
        const unsigned grid = static_cast<unsigned>(bwd_ctas(a.T, a.H, a.V, a.per_head));
        if (a.b) gn_bwd_kernel<X, kVec, NV, kBlock, true><<<grid, kThreads, smem, s>>>(a);
        else gn_bwd_kernel<X, kVec, NV, kBlock, false><<<grid, kThreads, smem, s>>>(a);
    } else {
        int64_t grid = std::min<int64_t>((a.T * a.H + groups - 1) / groups, 152 * 8);
        if (a.per_head) grid = (grid + a.H - 1) / a.H * a.H;
        else grid = std::max<int64_t>(grid, (a.H + groups - 1) / groups);
        gn_fwd_kernel<X, kVec, NV, kBlock><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
    }
    return launched();
}

// nv rounded up to what is compiled.
template <typename X, int kVec>
la_status by_row(Args& a, bool bwd, cudaStream_t s) {
    const Shape r = shape(a.V, kVec);
    constexpr int kMost = kPerLane / kVec;
    a.lanes = r.lanes;
    if (r.lanes == kThreads) return launch<X, kVec, kMost, true>(a, bwd, s);
    if (r.nv <= kMost / 4) return launch<X, kVec, kMost / 4, false>(a, bwd, s);
    return launch<X, kVec, kMost, false>(a, bwd, s);
}

template <typename X>
la_status dispatch(Args& a, bool bwd, cudaStream_t s) {
    auto fits = [&](int bytes) {
        const int n = bytes / static_cast<int>(sizeof(X));
        if (a.V % n) return false;
        auto ok = [&](const void* p, int64_t st, int64_t sh) {
            return !p || (aligned_to(p, bytes) && (a.T == 1 || st % n == 0) && (a.H == 1 || sh % n == 0));
        };
        return ok(a.x, a.x_st, a.x_sh) && ok(a.z, a.z_st, a.z_sh) && ok(a.dy, a.dy_st, a.dy_sh) && ok(a.y, a.y_st, a.y_sh) &&
               ok(a.dz, a.dz_st, a.dz_sh);
    };
    constexpr int kWide = 16 / static_cast<int>(sizeof(X));
    if (fits(16)) return by_row<X, kWide>(a, bwd, s);
    if (sizeof(X) == 2 && fits(8)) return by_row<X, 4>(a, bwd, s);
    return by_row<X, 1>(a, bwd, s);
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
    return (static_cast<size_t>(bwd_ctas(T, H, V, per_head != 0)) * V * 2 * 4 + 255) & ~size_t(255);
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
    a.T = p->T; a.H = p->H; a.V = p->V;
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
    a.T = p->T; a.H = p->H; a.V = p->V;
    a.per_head = p->per_head != 0; a.center = p->center != 0; a.act = p->activation; a.eps = p->eps;
    a.y = p->dx; a.y_st = p->dx_stride_t; a.y_sh = p->dx_stride_h;
    a.dz = p->dz; a.dz_st = p->dz_stride_t; a.dz_sh = p->dz_stride_h;
    int64_t ctas = bwd_ctas(a.T, a.H, a.V, a.per_head);
    a.pw = static_cast<float*>(p->workspace);
    a.pb = p->bias ? a.pw + ctas * a.V : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->T > 0) {
        st = p->x_dtype == LA_DTYPE_BF16 ? dispatch<bf16>(a, true, s) : dispatch<float>(a, true, s);
        if (st != LA_OK) return st;
    } else {
        ctas = 0;  // no rows: the sums are zero
    }
    const int heads = a.per_head ? a.H : 1;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.V) * heads + 31) / 32), a.pb ? 2 : 1);
    gn_sum_kernel<<<grid, 1024, 0, s>>>(a.pw, a.pb, ctas, a.V, heads, p->d_weight, p->d_bias, a.w_bf16);
    return launched();
}

}  // extern "C"
