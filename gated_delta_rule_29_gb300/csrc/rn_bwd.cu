// rn_bwd.cu -- the residual norm's backward (rn.cuh has the method).
#include "rn.cuh"

namespace la {
namespace rn {
namespace {

// CTAs of 256 threads that an SM holds, with room for the next row: 65536 x 4096 with an fp32 stream takes 671 us with one, 696
// with two (and spills), 692 with three and no row ahead; a floor of 641.
template <typename R, int kVec, int kElements>
constexpr int resident() { return kElements > 16 ? 1 : kVec == 1 ? (kElements > 8 ? 2 : 3) : kElements > 8 ? (sizeof(R) == 4 ? 1 : 2) : sizeof(R) == 4 ? 2 : 3; }
constexpr int kMostResident = 3;

// The weight gradient is summed in registers over kRows of a warp's rows at a time, those sums in shared memory (each word by one
// thread alone), then over the CTA's groups, then by a second launch over the CTAs, in an order fixed by the shape.  One running sum
// over a warp's rows was 435 units of 2^-24 off over 262144 equal rows (16-bit stream, 65536 x 4096: 325 us, now 328).
constexpr int kRows = 64;

template <typename X, typename R, int kVec, int NV, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, (resident<R, kVec, NV * kVec>())) rn_bwd_kernel(const Args a) {
    constexpr int P = NV * kVec / 2;
    __shared__ float2 red[2][32];
    extern __shared__ float sums[];  // [groups][V]
    const int warp = threadIdx.x >> 5;
    const int groups = (blockDim.x >> 5) / a.warps, g = warp / a.warps;
    const auto pl = place<kVec, NV>(warp % a.warps);
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups, rounds = (a.T + step - 1) / step;
    const float inv_v = 1.f / a.V;
    Vec<R, kVec> s[NV], dr[NV], next_s[NV], next_dr[NV];
    Vec<X, kVec> dy[NV], next_dy[NV];
    auto load = [&](Vec<R, kVec> (&to_s)[NV], Vec<X, kVec> (&to_dy)[NV], Vec<R, kVec> (&to_dr)[NV], int64_t t) {
        load_row<R, kVec, NV>(to_s, a.x, t * a.x_st, t < a.T, pl, a.V);
        load_row<X, kVec, NV>(to_dy, a.dy, t * a.dy_st, t < a.T, pl, a.V);
        if (a.dres) load_row<R, kVec, NV>(to_dr, a.dres, t * a.dres_st, t < a.T, pl, a.V);
    };
    constexpr bool kAhead = kVec > 1 && NV * kVec <= 16;
    int64_t t = static_cast<int64_t>(blockIdx.x) * groups + g;
    if (kAhead) load(next_s, next_dy, next_dr, t);
    constexpr bool kKeep = NV * kVec <= 16;
    float2 w[kKeep ? P : 1], dw[P];  // the weights are kept where a lane holds few elements
#pragma unroll
    for (int j = 0; j < (kKeep ? P : 0); ++j) w[j] = weight_pair<kVec, NV>(a, pl, j);
    auto weight = [&](int j) { return kKeep ? w[j] : weight_pair<kVec, NV>(a, pl, j); };
    auto each = [&](auto f) {  // f(word of this thread's column in sums, its place in dw)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (pl.column(k) + i < a.V) f(sums[g * a.V + pl.column(k) + i], k * kVec + i);
    };
    each([](float& word, int) { word = 0.f; });
    for (int64_t n = 0; n < rounds;) {
#pragma unroll
        for (int j = 0; j < P; ++j) dw[j] = both(0.f);
        for (const int64_t end = min(rounds, n + kRows); n < end; ++n, t += step) {
            const bool live = t < a.T;
            if (kAhead) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    s[k] = next_s[k];
                    dy[k] = next_dy[k];
                    dr[k] = next_dr[k];
                }
                load(next_s, next_dy, next_dr, t + step);
            } else {
                load(s, dy, dr, t);
            }
            float2 sq = both(0.f), sd = both(0.f);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 v = pair_of<R, kVec, NV>(s, j);
                sq = fma2(v, v, sq);
                sd = fma2(mul2(pair_of<X, kVec, NV>(dy, j), weight(j)), v, sd);
            }
            float sum = sq.x + sq.y, dot = sd.x + sd.y;
            row_reduce<false>(sum, dot, a.warps, red, static_cast<int>(n));
            const float rs = inv_sqrt(fmaf(sum, inv_v, a.eps)), m = -(dot * inv_v * rs * rs);  // mean(dn n) r, what s is taken off with
            if (!live) continue;  // a warp has one row
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 v = pair_of<R, kVec, NV>(s, j), d = pair_of<X, kVec, NV>(dy, j);
                dw[j] = fma2(d, mul2(v, both(rs)), dw[j]);
                float2 o = mul2(both(rs), fma2(v, both(m), mul2(d, weight(j))));
                if (a.dres) o = add2(o, pair_of<R, kVec, NV>(dr, j));
                set_pair<X, kVec, NV>(dy, j, o);
                set_pair<R, kVec, NV>(s, j, o);
            }
            if (a.y) store_row<X, kVec, NV>(a.y, t * a.y_st, dy, pl, a.V);
            if (a.ds) store_row<R, kVec, NV>(a.ds, t * a.ds_st, s, pl, a.V);
        }
        each([&](float& word, int e) { word += e % 2 ? dw[e / 2].y : dw[e / 2].x; });
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.V; c += blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < groups; ++q) s += sums[q * a.V + c];
        a.pw[static_cast<int64_t>(blockIdx.x) * a.V + c] = s;
    }
}

// dw[c] = the sum of the CTAs' partial sums.  A CTA takes 32 columns; its 32 warps take every 32nd row, in order.
__global__ void __launch_bounds__(1024) rn_sum_kernel(const float* pw, int64_t rows, int V, void* dw, int w_bf16) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = c < V ? strided_sum<16>(pw + c, V, w, rows, 32) : 0.f;
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < V) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += part[i][lane];
        store_any(dw, c, w_bf16, s);
    }
}

int64_t bwd_ctas(int64_t T, int V, int per_sm) {
    const Shape sh = shape(V);
    const int groups = sh.threads / 32 / sh.warps;
    return std::max<int64_t>(1, std::min<int64_t>((T + groups - 1) / groups, kSms * per_sm));
}

struct Launch {
    template <typename X, typename R, int kVec, int NV>
    static la_status run(Args& a, Shape sh, cudaStream_t s) {
        const size_t smem = static_cast<size_t>(sh.threads / 32 / sh.warps) * a.V * sizeof(float);
        a.ctas = bwd_ctas(a.T, a.V, resident<R, kVec, NV * kVec>());
        const unsigned grid = static_cast<unsigned>(a.ctas);
        if constexpr (NV * kVec == 32) {
            if (sh.threads == 512) {
                if (cudaFuncSetAttribute(rn_bwd_kernel<X, R, kVec, NV, 512>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxV * 4) != cudaSuccess) {
                    (void)cudaGetLastError();
                    return LA_ERR_CUDA;
                }
                rn_bwd_kernel<X, R, kVec, NV, 512><<<grid, 512, smem, s>>>(a);
                return launched();
            }
        }
        rn_bwd_kernel<X, R, kVec, NV, 256><<<grid, 256, smem, s>>>(a);
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

size_t la_rn_bwd_workspace_bytes(int64_t T, int32_t V) {
    if (T < 0 || V <= 0 || V > kMaxV) return 0;
    return (static_cast<size_t>(bwd_ctas(T, V, kMostResident)) * V * 4 + 255) & ~size_t(255);
}

la_status rn_bwd(const la_rn_bwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check(p->T, p->V, p->x_dtype, p->s_dtype, p->weight_dtype, p->eps, p->weight);
    if (st != LA_OK) return st;
    if (!good_rows(p->s, p->s_stride_t, p->T, p->V, p->s_dtype, false) || !good_rows(p->dy, p->dy_stride_t, p->T, p->V, p->x_dtype, false) ||
        (p->d_residual && !good_rows(p->d_residual, p->d_residual_stride_t, p->T, p->V, p->s_dtype, false)) ||
        (p->dx && !good_rows(p->dx, p->dx_stride_t, p->T, p->V, p->x_dtype, true)) ||
        (p->ds && !good_rows(p->ds, p->ds_stride_t, p->T, p->V, p->s_dtype, true)))
        return LA_ERR_INVALID_ARG;
    if ((p->T > 0 && !p->dx && !p->ds) || !p->d_weight || !aligned_to(p->d_weight, dtype_size(p->weight_dtype))) return LA_ERR_INVALID_ARG;
    const int xs = dtype_size(p->x_dtype), rs = dtype_size(p->s_dtype);
    auto over = [&](const void* out, int64_t st, int size) {
        return out && (clashes(out, st, size, p->s, p->s_stride_t, rs, p->T, p->V) || clashes(out, st, size, p->dy, p->dy_stride_t, xs, p->T, p->V) ||
                       clashes(out, st, size, p->d_residual, p->d_residual_stride_t, rs, p->T, p->V));
    };
    if (over(p->dx, p->dx_stride_t, xs) || over(p->ds, p->ds_stride_t, rs) ||
        (p->dx && p->ds && bytes_meet(p->dx, p->dx_stride_t * xs, int64_t(p->V) * xs, p->ds, p->ds_stride_t * rs, int64_t(p->V) * rs, p->T)))
        return LA_ERR_INVALID_ARG;
    if ((st = check_workspace(p->workspace, p->workspace_bytes, la_rn_bwd_workspace_bytes(p->T, p->V))) != LA_OK) return st;
    // the weight, which every row reads, and its gradient, which is written last
    const int64_t ws = dtype_size(p->weight_dtype) * int64_t(p->V);
    for (const void* w : {p->weight, static_cast<const void*>(p->d_weight)})
        if ((p->dx && bytes_meet(p->dx, p->dx_stride_t * xs, int64_t(p->V) * xs, w, 0, ws, p->T)) ||
            (p->ds && bytes_meet(p->ds, p->ds_stride_t * rs, int64_t(p->V) * rs, w, 0, ws, p->T)))
            return LA_ERR_INVALID_ARG;
    Args a = {};
    a.x = p->s; a.x_st = p->s_stride_t; a.dy = p->dy; a.dy_st = p->dy_stride_t; a.dres = p->d_residual; a.dres_st = p->d_residual_stride_t;
    a.w = p->weight; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.T = p->T; a.V = p->V; a.eps = p->eps;
    a.y = p->dx; a.y_st = p->dx_stride_t; a.ds = p->ds; a.ds_st = p->ds_stride_t;
    a.pw = static_cast<float*>(p->workspace);
    const int vec = 16 / xs;
    const bool wide = a.V % vec == 0 && wide_rows(a.x, a.x_st, rs, vec) && wide_rows(a.dy, a.dy_st, xs, vec) && wide_rows(a.dres, a.dres_st, rs, vec) &&
                      wide_rows(a.y, a.y_st, xs, vec) && wide_rows(a.ds, a.ds_st, rs, vec);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->T > 0 && (st = dispatch<Launch>(a, p->x_dtype, p->s_dtype, wide, s)) != LA_OK) return st;
    rn_sum_kernel<<<static_cast<unsigned>((a.V + 31) / 32), 1024, 0, s>>>(a.pw, a.ctas, a.V, p->d_weight, a.w_bf16);
    return launched();
}

}  // extern "C"
