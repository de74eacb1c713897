// rn.cuh -- the root-mean-square norm of whole rows with the residual's addition (rn_fwd, rn_bwd): what rn_fwd.cu and
// rn_bwd.cu share.
//
//   s = x + residual, rounded to the residual's type (the stream that goes on);  r = 1 / sqrt(mean(s^2) + eps),
//   n = s r,  y = n w, in the input's type or in 8 bits with scales;
//   dn = dy w,  ds = r (dn - n mean(dn n)) + d_residual,  dw = sum dy n.
//
// A row is spread over one to sixteen warps and stays in their registers: every operand is read once and every result
// written once, 16 bytes a lane where the rows' alignment allows.  Warp v of a row has the kSpan columns from v kSpan on,
// lane l of it kVec of them from (32 k + l) kVec on: the lanes that share a block of 32 or 128 columns then share a warp.
#pragma once
#include <algorithm>

#include "mixer.cuh"

namespace la {
namespace rn {

using namespace la::mixer;

constexpr int kMaxV = 16384;
constexpr int kSms = 152;

struct Args {
    const void *x, *res, *w, *dy, *dres;
    int64_t x_st, res_st, dy_st, dres_st, y_st, out_st, ds_st;
    int64_t T;
    int V, w_bf16, quant, blocks;  // scale blocks a row
    int warps;                     // of a row
    float eps;
    void *y, *out, *scales, *ds;   // y: the result, or dx in the backward; out: the sum
    float* pw;                     // partial sums [CTAs][V] of dw
    int64_t ctas;                  // of the backward (0 without rows: the sums are then zero)
};

// kVec consecutive elements in accesses of up to 16 bytes.
template <typename X, int kVec>
struct Vec {
    static constexpr int kPer = kVec * static_cast<int>(sizeof(X)) > 16 ? 16 / static_cast<int>(sizeof(X)) : kVec, kParts = kVec / kPer;
    Packed<X, kPer> p[kParts];
    __device__ __forceinline__ void load(const X* from) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) p[i].load(from + i * kPer);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kParts; ++i) p[i].zero();
    }
    __device__ __forceinline__ float get(int i) const { return p[i / kPer].get(i % kPer); }
    __device__ __forceinline__ void store(X* to) const {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            uint32_t* t = reinterpret_cast<uint32_t*>(to + i * kPer);
            const uint32_t* w = p[i].w;
            constexpr int kBytes = kPer * static_cast<int>(sizeof(X));
            if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(t) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(t) = make_uint2(w[0], w[1]);
            else if constexpr (kBytes == 4) *t = w[0];
            else *reinterpret_cast<uint16_t*>(t) = static_cast<uint16_t>(w[0]);
        }
    }
};
// Elements 2j and 2j + 1 of a lane's NV vectors, and the same rounded to X.
template <typename X, int kVec, int NV>
__device__ __forceinline__ float2 pair_of(const Vec<X, kVec> (&v)[NV], int j) {
    return make_float2(v[2 * j / kVec].get(2 * j % kVec), v[(2 * j + 1) / kVec].get((2 * j + 1) % kVec));
}
template <typename X, int kVec, int NV>
__device__ __forceinline__ void set_pair(Vec<X, kVec> (&v)[NV], int j, float2 f) {
    constexpr int kPer = Vec<X, kVec>::kPer;
    const int a = 2 * j % kVec, b = (2 * j + 1) % kVec;
    if constexpr (sizeof(X) == 4) {
        v[2 * j / kVec].p[a / kPer].w[a % kPer] = __float_as_uint(f.x);
        v[(2 * j + 1) / kVec].p[b / kPer].w[b % kPer] = __float_as_uint(f.y);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
        if constexpr (kVec == 1) {
            v[2 * j].p[0].w[0] = u & 0xFFFFu;
            v[2 * j + 1].p[0].w[0] = u >> 16;
        } else {
            v[2 * j / kVec].p[a / kPer].w[a % kPer / 2] = u;
        }
    }
}

template <int kVec, int NV>
struct Place {
    static constexpr int kSpan = 32 * kVec * NV;  // columns of a warp
    int base;
    __device__ __forceinline__ int column(int k) const { return base + 32 * kVec * k; }
};
template <int kVec, int NV>
__device__ __forceinline__ Place<kVec, NV> place(int warp_of_row) {
    return {warp_of_row * Place<kVec, NV>::kSpan + static_cast<int>(threadIdx.x & 31) * kVec};
}

template <typename X, int kVec, int NV>
__device__ __forceinline__ void load_row(Vec<X, kVec> (&v)[NV], const void* base, int64_t at, bool live, Place<kVec, NV> pl, int V) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = pl.column(k);
        if (live && c < V) v[k].load(static_cast<const X*>(base) + at + c);
        else v[k].zero();
    }
}
template <typename X, int kVec, int NV>
__device__ __forceinline__ void store_row(void* base, int64_t at, const Vec<X, kVec> (&v)[NV], Place<kVec, NV> pl, int V) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = pl.column(k);
        if (c < V) v[k].store(static_cast<X*>(base) + at + c);
    }
}
template <int kVec, int NV>
__device__ __forceinline__ float2 weight_pair(const Args& a, Place<kVec, NV> pl, int j) {
    const int c0 = pl.column(2 * j / kVec) + 2 * j % kVec, c1 = pl.column((2 * j + 1) / kVec) + (2 * j + 1) % kVec;
    return make_float2(c0 < a.V ? load_any(a.w, c0, a.w_bf16) : 0.f, c1 < a.V ? load_any(a.w, c1, a.w_bf16) : 0.f);
}

// The larger value, NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Over a row's warps: the sum of a, and the sum or (kMax) the largest of b.  red: [2][32] of float2, the halves taken in
// turn so that one barrier a row is enough.
template <bool kMax>
__device__ __forceinline__ void row_reduce(float& a, float& b, int warps, float2 (*red)[32], int turn) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        const float o = __shfl_xor_sync(0xffffffffu, b, off);
        b = kMax ? max_nan(b, o) : b + o;
    }
    if (warps == 1) return;
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[turn & 1][w] = make_float2(a, b);
    __syncthreads();
    const int first = w & ~(warps - 1);
    float2 t = red[turn & 1][first];
    for (int i = 1; i < warps; ++i) {
        const float2 o = red[turn & 1][first + i];
        t.x += o.x;
        t.y = kMax ? max_nan(t.y, o.y) : t.y + o.y;
    }
    a = t.x;
    b = t.y;
}

// 1 / sqrt(v) in 32 bits: the approximation and one step of Newton's method (where r^2 v is finite).
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r0 = rsqrtf(v), e = fmaf(-v * r0, r0, 1.f);
    return fabsf(e) < 0.5f ? fmaf(0.5f * r0, e, r0) : r0;
}

// How a row is spread: at most 16 elements a lane up to eight warps, then 32; sixteen warps beyond 8192.
struct Shape {
    int warps, each, threads;
};
inline Shape shape(int V) {
    Shape s = {1, 8, 256};
    if (V > 256) s.each = 16;
    while (s.warps < 8 && 32 * s.warps * s.each < V) s.warps *= 2;
    if (32 * s.warps * s.each < V) s.each = 32;
    if (32 * s.warps * s.each < V) {
        s.warps = 16;
        s.threads = 512;
    }
    return s;
}

// Launch::run<X, R, kVec, NV>: one row's vectors of 16 bytes of X, or single elements.
template <typename Launch, typename X, typename R>
la_status by_row(Args& a, bool wide, cudaStream_t s) {
    const Shape sh = shape(a.V);
    a.warps = sh.warps;
    constexpr int kWide = 16 / static_cast<int>(sizeof(X));
    if (wide) {
        if (sh.each == 8) return Launch::template run<X, R, kWide, 8 / kWide>(a, sh, s);
        if (sh.each == 16) return Launch::template run<X, R, kWide, 16 / kWide>(a, sh, s);
        return Launch::template run<X, R, kWide, 32 / kWide>(a, sh, s);
    }
    if (sh.each == 8) return Launch::template run<X, R, 1, 8>(a, sh, s);
    if (sh.each == 16) return Launch::template run<X, R, 1, 16>(a, sh, s);
    return Launch::template run<X, R, 1, 32>(a, sh, s);
}
template <typename Launch>
la_status dispatch(Args& a, int32_t xd, int32_t rd, bool wide, cudaStream_t s) {
    if (xd == LA_DTYPE_F32) return by_row<Launch, float, float>(a, wide, s);
    return rd == LA_DTYPE_F32 ? by_row<Launch, bf16, float>(a, wide, s) : by_row<Launch, bf16, bf16>(a, wide, s);
}

// Whether rows of V elements of `size` bytes take accesses of kVec elements, of at most 16 bytes each.  A single row asks for its
// stride too: wide rows sum in another order, and a row alone has the bits that it has among others.
inline bool wide_rows(const void* p, int64_t st, int64_t size, int vec) {
    const int64_t bytes = std::min<int64_t>(16, vec * size);
    return !p || (aligned_to(p, bytes) && st * size % bytes == 0);
}

inline la_status check(int64_t T, int32_t V, int32_t xd, int32_t rd, int32_t wd, float eps, const void* w) {
    if (T < 0 || V <= 0) return LA_ERR_INVALID_ARG;
    if (!known_dtype(xd) || !known_dtype(rd) || !known_dtype(wd) || (xd == LA_DTYPE_F32 && rd != LA_DTYPE_F32)) return LA_ERR_UNSUPPORTED;
    if (!(eps > 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    if (V > kMaxV || T >= (int64_t(1) << 40)) return LA_ERR_UNSUPPORTED;
    return w && aligned_to(w, dtype_size(wd)) ? LA_OK : LA_ERR_INVALID_ARG;
}

}  // namespace rn
}  // namespace la
