// gn.cuh -- group norm of every head's channels of every token, with an activation or a gate
// (gn_fwd, gn_bwd):
// what gn_fwd.cu and gn_bwd.cu share.
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
#pragma once
#include <algorithm>
#include <type_traits>

#include "mixer.cuh"

namespace la {
namespace gn {

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
    int64_t ctas;         // of the backward (0 without rows: the sums are then zero)
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

// Resident CTAs to compile for: more, with fewer registers each, where a lane holds little.  A launch takes one wave of
// them: a part of a second one leaves SMs idle, a whole second one starts over for nothing.  Forward, gated 65536 x 32 x
// 128: bf16 (four an SM) 258 us with 4 x 152 CTAs, 287 with 3, 293 with 6; fp32 a quarter of that (three) 125 with 3,
// 143 with 4; 16384 x 16 x 512 (two) 211 with 2, 262 with 3.  Backward: bf16 (three) 440 with 3 x 152, 498 with 2, 549 with
// 4; with a bias (two) 471 with 2, 563 with 3, 479 with 6; 16384 x 16 x 512 (one) 438 with 1, 457 with 6; and the fewer
// the CTAs, the fewer the partial sums.
constexpr int kSms = 152;
constexpr int ctas(int elements, int few, int many) { return elements <= 8 ? many : elements <= 16 ? few : 1; }

// ---------------------------------------------------------------- shapes
// How a row is spread over lanes: vectors of 16 bytes, of 8 (bf16), pairs or single elements; as few lanes as hold it at 8
// elements each, up to a warp (the fewer lanes, the fewer shuffles a row), then up to kPerLane elements a lane, then
// the whole CTA.
constexpr int kPerLane = 32;

struct Shape {
    int lanes, nv;
};
inline Shape shape(int V, int vec) {
    const int n = (V + vec - 1) / vec;  // vectors
    Shape s = {1, 1};
    while (s.lanes < 32 && s.lanes * (8 / vec) < n) s.lanes *= 2;
    if (V > 32 * kPerLane) s.lanes = kThreads;
    s.nv = (n + s.lanes - 1) / s.lanes;
    return s;
}

// Launch::run<X, kVec, NV, kBlock> for the row's spread, nv rounded up to what is compiled.
template <typename Launch, typename X, int kVec>
la_status by_row(Args& a, cudaStream_t s) {
    const Shape r = shape(a.V, kVec);
    constexpr int kMost = kPerLane / kVec;
    a.lanes = r.lanes;
    if (r.lanes == kThreads) return Launch::template run<X, kVec, kMost, true>(a, s);
    if (r.nv <= kMost / 4) return Launch::template run<X, kVec, kMost / 4, false>(a, s);
    if (r.nv <= kMost / 2) return Launch::template run<X, kVec, kMost / 2, false>(a, s);
    return Launch::template run<X, kVec, kMost, false>(a, s);
}

template <typename Launch, typename X>
la_status dispatch(Args& a, cudaStream_t s) {
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
    if (fits(16)) return by_row<Launch, X, kWide>(a, s);
    if (sizeof(X) == 2 && fits(8)) return by_row<Launch, X, 4>(a, s);
    if (fits(2 * sizeof(X))) return by_row<Launch, X, 2>(a, s);
    return by_row<Launch, X, 1>(a, s);
}

// Whether the T x H rows of V elements, st and sh elements apart, share no memory.
inline bool rows_apart(int64_t st, int64_t sh, int64_t T, int64_t H, int64_t V) {
    if (T == 1 || H == 1) return T * H == 1 || (T == 1 ? sh : st) >= V;
    const bool by_head = sh <= st;
    const int64_t a = by_head ? sh : st, na = by_head ? H : T, b = by_head ? st : sh, nb = by_head ? T : H;  // a <= b
    if (a < V) return false;
    // row j b lies among the na rows that are a apart, or beyond the last of them
    for (int64_t j = 1; j < nb && j * b / a < na; ++j) {
        const int64_t q = j * b / a, r = j * b % a;
        if (r < V || (a - r < V && q + 1 < na)) return false;
    }
    return true;
}

inline bool good_thd(const void* p, int64_t st, int64_t sh, int64_t T, int H, int V, int32_t dtype, bool out) {
    if (T == 0) return true;
    if (!p || !aligned_to(p, dtype_size(dtype)) || st < 0 || sh < 0) return false;
    return !out || rows_apart(st, sh, T, H, V);
}

inline la_status check(int64_t T, int H, int V, int32_t xd, int32_t wd, int32_t act, float eps, const void* w, const void* b) {
    if (T < 0 || H <= 0 || V <= 0) return LA_ERR_INVALID_ARG;
    if (!known_dtype(xd) || !known_dtype(wd)) return LA_ERR_UNSUPPORTED;
    if (act < LA_ACT_NONE || act > LA_ACT_SIGMOID) return LA_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    if (V > kMaxV || T >= (int64_t(1) << 40) / H) return LA_ERR_UNSUPPORTED;
    if (!w || !aligned_to(w, dtype_size(wd)) || !good_optional(b, wd)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

}  // namespace gn
}  // namespace la
