// rn_fwd.cu -- the residual norm's forward (rn.cuh has the method).
#include "rn.cuh"

namespace la {
namespace rn {
namespace {

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int kVec>
__device__ __forceinline__ void store_e4m3(uint8_t* to, const float2* v, int k) {
    if constexpr (kVec == 1) {
        *to = static_cast<uint8_t>(e4m3_pair(k % 2 ? v->y : v->x, 0.f));
    } else {
        uint32_t w[kVec / 4];
#pragma unroll
        for (int i = 0; i < kVec / 4; ++i) w[i] = e4m3_pair(v[2 * i].x, v[2 * i].y) | e4m3_pair(v[2 * i + 1].x, v[2 * i + 1].y) << 16;
        if constexpr (kVec == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(to) = w[0];
    }
}

constexpr float kTop = 448.f;  // the largest e4m3 value

// A block's scale from its largest |y|, which counts as 2^-100 at least: most / 448, or as a power of two the least with
// most <= 448 scale: with most = m 2^e, 1 <= m < 2, that is 2^(e - 8), or 2^(e - 7) where m > 1.75.
struct Scale {
    float inverse;
    float scale;
    uint8_t exponent;  // of the power of two, as e8m0 has it; 255 (NaN) where most is not finite
};
// Where most is not finite all three are NaN, and with them the block's values.
__device__ __forceinline__ Scale scale_of(float most, bool power) {
    most = max_nan(most, 0x1p-100f);
    Scale s;
    if (power) {
        const uint32_t b = __float_as_uint(most), e = (b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);
        s.exponent = b >= 0x7F800000u ? 255 : static_cast<uint8_t>(e);
        s.scale = __uint_as_float(b >= 0x7F800000u ? 0x7FC00000u : e << 23);
        s.inverse = __uint_as_float(b >= 0x7F800000u ? 0x7FC00000u : (254u - e) << 23);
    } else {
        s.exponent = 0;
        most = fmaf(most, 0.f, most);  // itself, or NaN
        s.scale = __fdiv_rn(most, kTop);
        s.inverse = __fdiv_rn(kTop, most);
    }
    return s;
}

// CTAs of 256 threads that an SM holds.
template <typename R, int kVec, int kElements>
constexpr int resident() { return kElements > 16 ? 1 : kVec == 1 ? 4 : kElements > 8 ? (sizeof(R) == 4 ? 2 : 3) : sizeof(R) == 4 ? 3 : 4; }

template <typename X, typename R, int kVec, int NV, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, (resident<R, kVec, NV * kVec>())) rn_fwd_kernel(const Args a) {
    constexpr int P = NV * kVec / 2;
    __shared__ float2 red[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (blockDim.x >> 5) / a.warps, g = warp / a.warps;
    const auto pl = place<kVec, NV>(warp % a.warps);
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups, rounds = (a.T + step - 1) / step;
    const float inv_v = 1.f / a.V;
    Vec<X, kVec> x[NV], next_x[NV];
    Vec<R, kVec> r[NV], next_r[NV];
    auto load = [&](Vec<X, kVec> (&to_x)[NV], Vec<R, kVec> (&to_r)[NV], int64_t t) {
        load_row<X, kVec, NV>(to_x, a.x, t * a.x_st, t < a.T, pl, a.V);
        if (a.res) load_row<R, kVec, NV>(to_r, a.res, t * a.res_st, t < a.T, pl, a.V);
    };
    // the next row is on its way while this one is worked on, where a lane holds few elements (65536 x 4096 to 8 bits: 349 us,
    // 30 % more without; a floor of 281)
    constexpr bool kAhead = kVec > 1 && NV * kVec <= 16;
    int64_t t = static_cast<int64_t>(blockIdx.x) * groups + g;
    if (kAhead) load(next_x, next_r, t);
    constexpr bool kKeep = NV * kVec <= 16;
    float2 w[kKeep ? P : 1];  // kept where a lane holds few elements
#pragma unroll
    for (int j = 0; j < (kKeep ? P : 0); ++j) w[j] = weight_pair<kVec, NV>(a, pl, j);
    for (int64_t n = 0; n < rounds; ++n, t += step) {
        const bool live = t < a.T;
        if (kAhead) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                x[k] = next_x[k];
                r[k] = next_r[k];
            }
            load(next_x, next_r, t + step);
        } else {
            load(x, r, t);
        }
        float2 s[P], sq = both(0.f);
        if (a.res) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                set_pair<R, kVec, NV>(r, j, add2(pair_of<X, kVec, NV>(x, j), pair_of<R, kVec, NV>(r, j)));
                s[j] = pair_of<R, kVec, NV>(r, j);
            }
            if (live) store_row<R, kVec, NV>(a.out, t * a.out_st, r, pl, a.V);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = pair_of<X, kVec, NV>(x, j);
        }
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            sq = fma2(s[j], s[j], sq);
            s[j] = mul2(s[j], kKeep ? w[j] : weight_pair<kVec, NV>(a, pl, j));
            if (a.quant == LA_QUANT_ROW) most = max_nan(most, max_nan(fabsf(s[j].x), fabsf(s[j].y)));
        }
        float sum = sq.x + sq.y;
        row_reduce<true>(sum, most, a.warps, red, static_cast<int>(n));
        float rs = inv_sqrt(fmaf(sum, inv_v, a.eps));
        if (!live) continue;  // a warp has one row
        if (a.quant == LA_QUANT_NONE) {
#pragma unroll
            for (int j = 0; j < P; ++j) set_pair<X, kVec, NV>(x, j, mul2(s[j], both(rs)));
            store_row<X, kVec, NV>(a.y, t * a.y_st, x, pl, a.V);
            continue;
        }
        // y / scale as s w times (r / scale): a block's largest |y| is its largest |s w| times r.  The factor is 448 r / 2^-100 at
        // most, within the range up to r = 2^19; beyond (rows of 2e-6 and less, padding, under a small eps) s w takes r first
        // (65536 x 4096 in blocks of 32: 343 us without that question, 349 with it, by block 361 and 366, by row 337 and 340; as a
        // second copy of the code below the same, but odd rows 201 -> 210).
        if (rs > 0x1p19f) {
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = mul2(s[j], both(rs));
            most *= rs;
            rs = 1.f;
        }
        if (a.quant == LA_QUANT_ROW) {
            const Scale sc = scale_of(most * rs, false);
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = mul2(s[j], both(rs * sc.inverse));
            if (warp % a.warps == 0 && lane == 0) static_cast<float*>(a.scales)[t] = sc.scale;
        } else {
            // a block is kLanes lanes of kParts vectors
            auto blocks = [&](auto width) {
                constexpr int kLanes = width / kVec < 32 ? width / kVec : 32, kParts = width / kVec < 32 ? 1 : width / kVec / 32;
#pragma unroll
                for (int k = 0; k < NV; k += kParts) {
                    float m = 0.f;
#pragma unroll
                    for (int e = k * kVec; e < (k + kParts) * kVec; ++e) m = max_nan(m, fabsf(e % 2 ? s[e / 2].y : s[e / 2].x));
#pragma unroll
                    for (int off = 1; off < kLanes; off *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
                    const Scale sc = scale_of(m * rs, width == 32);
                    const float f = rs * sc.inverse;
#pragma unroll
                    for (int e = k * kVec; e < (k + kParts) * kVec; ++e) (e % 2 ? s[e / 2].y : s[e / 2].x) *= f;
                    const int c = pl.column(k);
                    if (c < a.V && lane % kLanes == 0) {
                        const int64_t at = t * a.blocks + c / width;
                        if (width == 32) static_cast<uint8_t*>(a.scales)[at] = sc.exponent;
                        else static_cast<float*>(a.scales)[at] = sc.scale;
                    }
                }
            };
            if (a.quant == LA_QUANT_MX) blocks(std::integral_constant<int, 32>());
            else blocks(std::integral_constant<int, 128>());
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = pl.column(k);
            if (c < a.V) store_e4m3<kVec>(static_cast<uint8_t*>(a.y) + t * a.y_st + c, s + k * kVec / 2, k);
        }
    }
}

struct Launch {
    template <typename X, typename R, int kVec, int NV>
    static la_status run(const Args& a, Shape sh, cudaStream_t s) {
        const int groups = sh.threads / 32 / sh.warps;
        const int64_t grid = std::min<int64_t>((a.T + groups - 1) / groups, kSms * resident<R, kVec, NV * kVec>());
        if constexpr (NV * kVec == 32) {
            if (sh.threads == 512) {
                rn_fwd_kernel<X, R, kVec, NV, 512><<<static_cast<unsigned>(grid), 512, 0, s>>>(a);
                return launched();
            }
        }
        rn_fwd_kernel<X, R, kVec, NV, 256><<<static_cast<unsigned>(grid), 256, 0, s>>>(a);
        return launched();
    }
};

}  // namespace
}  // namespace rn
}  // namespace la

using namespace la;
using namespace la::mixer;
using namespace la::rn;

extern "C" {

int32_t la_rn_scale_blocks(int32_t V, int32_t quantize) {
    if (V <= 0) return 0;
    return quantize == LA_QUANT_ROW ? 1 : quantize == LA_QUANT_BLOCK ? (V - 1) / 128 + 1 : quantize == LA_QUANT_MX ? (V - 1) / 32 + 1 : 0;
}

la_status rn_fwd(const la_rn_fwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    const int32_t rd = p->residual ? p->residual_dtype : p->x_dtype;
    la_status st = check(p->T, p->V, p->x_dtype, rd, p->weight_dtype, p->eps, p->weight);
    if (st != LA_OK) return st;
    if (p->quantize < LA_QUANT_NONE || p->quantize > LA_QUANT_MX) return LA_ERR_INVALID_ARG;
    const bool eight = p->quantize != LA_QUANT_NONE;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->V, p->x_dtype, false)) return LA_ERR_INVALID_ARG;
    if (p->residual && (!good_rows(p->residual, p->residual_stride_t, p->T, p->V, rd, false) ||
                        !good_rows(p->residual_out, p->residual_out_stride_t, p->T, p->V, rd, true)))
        return LA_ERR_INVALID_ARG;
    if (p->T > 0 && (!p->y || p->y_stride_t < 0 || (p->T > 1 && p->y_stride_t < p->V) || (!eight && !aligned_to(p->y, dtype_size(p->x_dtype)))))
        return LA_ERR_INVALID_ARG;
    if (eight && p->T > 0 && (!p->scales || (p->quantize != LA_QUANT_MX && !aligned_to(p->scales, 4)))) return LA_ERR_INVALID_ARG;
    const int64_t xs = dtype_size(p->x_dtype), ss = dtype_size(rd), ys = eight ? 1 : xs;
    if (clashes(p->y, p->y_stride_t, ys, p->x, p->x_stride_t, xs, p->T, p->V)) return LA_ERR_INVALID_ARG;
    if (p->residual && (clashes(p->y, p->y_stride_t, ys, p->residual, p->residual_stride_t, ss, p->T, p->V) ||
                        clashes(p->residual_out, p->residual_out_stride_t, ss, p->x, p->x_stride_t, xs, p->T, p->V) ||
                        clashes(p->residual_out, p->residual_out_stride_t, ss, p->residual, p->residual_stride_t, ss, p->T, p->V) ||
                        bytes_meet(p->y, p->y_stride_t * ys, p->V * ys, p->residual_out, p->residual_out_stride_t * ss, p->V * ss, p->T)))
        return LA_ERR_INVALID_ARG;
    // the weight, which every row reads, and the scales: one row, and rows of their own
    const int64_t ws = dtype_size(p->weight_dtype), cs = int64_t(la_rn_scale_blocks(p->V, p->quantize)) * (p->quantize == LA_QUANT_MX ? 1 : 4);
    auto on = [&](const void* q, int64_t st, int64_t size, const void* r, int64_t r_st, int64_t r_row) {
        return q && r && bytes_meet(q, st * size, p->V * size, r, r_st, r_row, p->T);
    };
    const void *out = p->residual ? p->residual_out : nullptr, *scales = eight ? p->scales : nullptr;
    if (on(p->y, p->y_stride_t, ys, p->weight, 0, p->V * ws) || on(out, p->residual_out_stride_t, ss, p->weight, 0, p->V * ws) ||
        on(p->y, p->y_stride_t, ys, scales, cs, cs) || on(out, p->residual_out_stride_t, ss, scales, cs, cs) ||
        on(p->x, p->x_stride_t, xs, scales, cs, cs) || on(p->residual, p->residual_stride_t, ss, scales, cs, cs) ||
        (scales && bytes_meet(p->weight, 0, p->V * ws, scales, cs, cs, p->T)))
        return LA_ERR_INVALID_ARG;
    if (p->T == 0) return LA_OK;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.res = p->residual; a.res_st = p->residual_stride_t;
    a.w = p->weight; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.T = p->T; a.V = p->V; a.eps = p->eps; a.quant = p->quantize; a.blocks = la_rn_scale_blocks(p->V, p->quantize);
    a.y = p->y; a.y_st = p->y_stride_t; a.out = p->residual ? p->residual_out : nullptr; a.out_st = p->residual_out_stride_t;
    a.scales = p->scales;
    const int vec = 16 / static_cast<int>(xs);
    const bool wide = a.V % vec == 0 && wide_rows(a.x, a.x_st, xs, vec) && wide_rows(a.res, a.res_st, ss, vec) &&
                      wide_rows(a.out, a.out_st, ss, vec) && wide_rows(a.y, a.y_st, ys, vec);
    return dispatch<Launch>(a, p->x_dtype, rd, wide, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
