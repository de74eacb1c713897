// gn_fwd.cu -- the group norm's forward (gn.cuh has the method).
#include "gn.cuh"

namespace la {
namespace gn {
namespace {

template <typename X, int kVec, int NV>
constexpr int resident() { return ctas(NV * kVec, 2, sizeof(X) == 4 || kVec < 4 ? 3 : 4); }

// Bound by its bytes (2 rows, 3 with a gate): 65536 x 32 x 128 bf16, gated, in 256 us, 6.3 TB/s (94 % of the measured
// copy rate).  A single row a group at a time leaves too little in flight, so short rows are requested one ahead.
template <typename X, int kVec, int NV, bool kBlock>
__global__ void __launch_bounds__(kThreads, (resident<X, kVec, NV>())) gn_fwd_kernel(const Args a) {
    __shared__ float red[kThreads / 32];
    const int lane = threadIdx.x % a.lanes;
    const Walk r = walk(a);
    const int64_t rounds = (a.T + r.step - 1) / r.step;  // the same for every lane of a warp: the shuffles need them all
    const float inv_v = 1.f / a.V;
    constexpr int kPairs = NV * kVec / 2;
    float2 w[kPairs], b[kPairs];
    Packed<X, kVec> raw[NV], z[NV], next[NV], next_z[NV];
    auto load = [&](Packed<X, kVec> (&x)[NV], Packed<X, kVec> (&g)[NV], int64_t t) {
        load_row<X, kVec, NV>(x, a.x, t * a.x_st + r.h * a.x_sh, t < a.T, lane, a);
        if (a.z) load_row<X, kVec, NV>(g, a.z, t * a.z_st + r.h * a.z_sh, t < a.T, lane, a);
    };
    // short rows: the next one is on its way while this one is worked on
    constexpr bool kAhead = NV * kVec <= 8 && kVec * sizeof(X) >= 8;
    int64_t t = r.t0;
    if (kAhead) load(next, next_z, t);
    load_weights<kVec, NV>(w, a.w, r.h, lane, a);
    load_weights<kVec, NV>(b, a.b, r.h, lane, a);
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

struct Launch {
    template <typename X, int kVec, int NV, bool kBlock>
    static la_status run(const Args& a, cudaStream_t s) {
        const int groups = kThreads / a.lanes;
        int64_t grid = std::min<int64_t>((a.T * a.H + groups - 1) / groups, kSms * resident<X, kVec, NV>());
        if (a.per_head) grid = (grid + a.H - 1) / a.H * a.H;
        else grid = std::max<int64_t>(grid, (a.H + groups - 1) / groups);
        gn_fwd_kernel<X, kVec, NV, kBlock><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
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
    return p->x_dtype == LA_DTYPE_BF16 ? dispatch<Launch, bf16>(a, s) : dispatch<Launch, float>(a, s);
}

}  // extern "C"
