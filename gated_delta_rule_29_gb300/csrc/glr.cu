// glr.cu -- the gated linear recurrence (glr_fwd, glr_bwd, glr_decode).
//
// Per sequence and channel, with l_t the log decay of g_t, a_t = e^{l_t} and m_t = 1 or 1 - a_t:
//
//   h_t = a_t h_{t-1} + m_t x_t
//
// and backwards, e_t being the gradient of h_t:
//
//   e_t = dh_t + a_{t+1} e_{t+1},  dx_t = m_t e_t,  dl_t = e_t a_t (h_{t-1} - [m = 1 - a] x_t),
//   dg_t = dl_t dl/dg,  d(initial) = a_1 e_1.
//
// The simplest form: one thread walks one channel of one sequence.
#include <algorithm>

#include "mixer.cuh"

namespace {

using namespace la::mixer;

constexpr int kBlock = 128;    // tokens between saved states
constexpr int kThreads = 128;

// a, m and dl/dg of one gate value.  The log sigmoid's a = s(g) and 1 - a = s(-g) come from
// e = exp(-|g|) without cancellation; otherwise 1 - a = -expm1(l).
__device__ __forceinline__ void gate(int mode, float lb, bool compl_in, float g, float& a, float& m, float& slope) {
    if (mode == LA_GATE_LOGSIGMOID) {
        const float e = expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
        a = g >= 0.f ? big : small;
        slope = g >= 0.f ? small : big;
        m = compl_in ? slope : 1.f;
        return;
    }
    float l = g;
    slope = 1.f;
    if (mode == LA_GATE_SIGMOID_BOUND) {
        const float e = expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
        l = lb * (g >= 0.f ? big : small);
        slope = l * (g >= 0.f ? small : big);
    }
    a = expf(l);
    m = compl_in ? -expm1f(l) : 1.f;
}

struct Args {
    const void *x, *g, *cu, *s0;
    int64_t x_st, g_st, T;
    int cu64, N, D, mode, compl_in, s0_bf16;
    float lb;
    const int32_t* idx;
    int64_t pool;
    void* h;
    int64_t h_st;
    float *fin, *ckpt;
    const void* dh;
    const float* dfin;
    void *dx, *dg;
    int64_t dh_st, dx_st, dg_st;
    float* ds0;
    int32_t* status;
};

// The tokens [lo, hi) of sequence i, or false (with the status set) when cu_seqlens is invalid.
__device__ bool sequence(const Args& a, int i, int64_t& lo, int64_t& hi) {
    lo = cu_load(a.cu, a.cu64, i);
    hi = cu_load(a.cu, a.cu64, i + 1);
    if (lo < 0 || hi < lo || hi > a.T || (i == 0 && lo != 0) || (i == a.N - 1 && hi != a.T)) {
        raise_status(a.status, LA_ERR_BAD_SEQLENS);
        return false;
    }
    return true;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) glr_fwd_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.N || d >= a.D) return;
    int64_t lo, hi;
    if (!sequence(a, i, lo, hi)) return;
    int64_t slot = i;
    if (a.idx) {
        slot = a.idx[i];
        if (slot < 0 || slot >= a.pool) {
            raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
            return;
        }
    }
    float h = a.s0 ? load_any(a.s0, slot * a.D + d, a.s0_bf16) : 0.f;
    for (int64_t t = lo; t < hi; ++t) {
        if (a.ckpt && (t - lo) % kBlock == 0) a.ckpt[(lo / kBlock + i + (t - lo) / kBlock) * a.D + d] = h;
        float dec, m, slope;
        gate(a.mode, a.lb, a.compl_in, to_f(static_cast<const G*>(a.g)[t * a.g_st + d]), dec, m, slope);
        h = fmaf(dec, h, m * to_f(static_cast<const X*>(a.x)[t * a.x_st + d]));
        if (a.h) static_cast<X*>(a.h)[t * a.h_st + d] = from_f<X>(h);
    }
    if (a.idx) store_any(const_cast<void*>(a.s0), slot * a.D + d, a.s0_bf16, h);
    else if (a.fin) a.fin[static_cast<int64_t>(i) * a.D + d] = h;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) glr_bwd_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.N || d >= a.D) return;
    int64_t lo, hi;
    if (!sequence(a, i, lo, hi)) return;
    float prev[kBlock];
    float e = a.dfin ? a.dfin[static_cast<int64_t>(i) * a.D + d] : 0.f;  // gradient of h_t from later tokens
    for (int64_t c = (hi - lo + kBlock - 1) / kBlock - 1; c >= 0; --c) {
        const int64_t t0 = lo + c * kBlock;
        const int n = static_cast<int>(min(static_cast<int64_t>(kBlock), hi - t0));
        float dec, m, slope, h = a.ckpt[(lo / kBlock + i + c) * a.D + d];
        for (int k = 0; k < n; ++k) {
            prev[k] = h;
            gate(a.mode, a.lb, a.compl_in, to_f(static_cast<const G*>(a.g)[(t0 + k) * a.g_st + d]), dec, m, slope);
            h = fmaf(dec, h, m * to_f(static_cast<const X*>(a.x)[(t0 + k) * a.x_st + d]));
        }
        for (int k = n - 1; k >= 0; --k) {
            const int64_t t = t0 + k;
            const float x = to_f(static_cast<const X*>(a.x)[t * a.x_st + d]);
            gate(a.mode, a.lb, a.compl_in, to_f(static_cast<const G*>(a.g)[t * a.g_st + d]), dec, m, slope);
            e += to_f(static_cast<const X*>(a.dh)[t * a.dh_st + d]);
            static_cast<X*>(a.dx)[t * a.dx_st + d] = from_f<X>(m * e);
            e *= dec;
            static_cast<G*>(a.dg)[t * a.dg_st + d] = from_f<G>(e * (a.compl_in ? prev[k] - x : prev[k]) * slope);
        }
    }
    if (a.ds0) a.ds0[static_cast<int64_t>(i) * a.D + d] = e;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) glr_decode_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.N || d >= a.D) return;
    int64_t slot = i;
    if (a.idx) {
        slot = a.idx[i];
        if (slot < 0 || slot >= a.pool) {
            raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
            return;
        }
    }
    float dec, m, slope;
    gate(a.mode, a.lb, a.compl_in, to_f(static_cast<const G*>(a.g)[i * a.g_st + d]), dec, m, slope);
    const float h = fmaf(dec, load_any(a.s0, slot * a.D + d, a.s0_bf16), m * to_f(static_cast<const X*>(a.x)[i * a.x_st + d]));
    store_any(const_cast<void*>(a.s0), slot * a.D + d, a.s0_bf16, h);
    static_cast<X*>(a.h)[i * a.h_st + d] = from_f<X>(h);
}

enum Which { kFwd, kBwd, kDecode };

template <typename X, typename G>
la_status launch(const Args& a, Which w, cudaStream_t s) {
    if (a.N == 0 || a.D == 0) return LA_OK;
    const unsigned ny = std::min(a.N, 65535), nz = (a.N + ny - 1) / ny;
    const dim3 grid((a.D + kThreads - 1) / kThreads, ny, nz);
    if (w == kFwd) glr_fwd_kernel<X, G><<<grid, kThreads, 0, s>>>(a);
    else if (w == kBwd) glr_bwd_kernel<X, G><<<grid, kThreads, 0, s>>>(a);
    else glr_decode_kernel<X, G><<<grid, kThreads, 0, s>>>(a);
    return launched();
}

la_status dispatch(const Args& a, int32_t xd, int32_t gd, Which w, cudaStream_t s) {
    if (xd == LA_DTYPE_BF16) return gd == LA_DTYPE_BF16 ? launch<bf16, bf16>(a, w, s) : launch<bf16, float>(a, w, s);
    return gd == LA_DTYPE_BF16 ? launch<float, bf16>(a, w, s) : launch<float, float>(a, w, s);
}

}  // namespace

extern "C" {

size_t la_glr_checkpoint_rows(int64_t T, int32_t N) {
    return T < 0 || N < 0 ? 0 : static_cast<size_t>(T / kBlock + N);
}

size_t la_glr_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t backward, int32_t checkpoints_given) {
    if (T < 0 || N < 0 || D < 0 || !backward || checkpoints_given) return 0;
    return (la_glr_checkpoint_rows(T, N) * D * 4 + 255) & ~size_t(255);
}

la_status glr_fwd(const la_glr_fwd_params* p, void* stream) {
    if (!p || p->D <= 0) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->g_dtype)) return LA_ERR_UNSUPPORTED;
    if (p->initial_state && !known_dtype(p->initial_state_dtype)) return LA_ERR_UNSUPPORTED;
    if ((st = check_gate(p->gate_mode, p->gate_lower_bound)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->g, p->g_stride_t, p->T, p->D, p->g_dtype, false) ||
        !good_rows(p->h, p->h_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_optional(p->initial_state, p->initial_state_dtype) || !good_optional(p->final_state, LA_DTYPE_F32) ||
        !good_optional(p->checkpoints, LA_DTYPE_F32))
        return LA_ERR_INVALID_ARG;
    if (p->state_indices && (!aligned_to(p->state_indices, 4) || !p->initial_state || p->final_state || p->state_pool_size <= 0))
        return LA_ERR_INVALID_ARG;
    if ((st = check_workspace(p->workspace, p->workspace_bytes, la_glr_workspace_bytes(p->T, p->N, p->D, 0, 0))) != LA_OK) return st;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.g = p->g; a.g_st = p->g_stride_t;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D;
    a.mode = p->gate_mode; a.lb = p->gate_lower_bound; a.compl_in = p->complement_input != 0;
    a.s0 = p->initial_state; a.s0_bf16 = p->initial_state_dtype == LA_DTYPE_BF16;
    a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.h = p->h; a.h_st = p->h_stride_t; a.fin = p->final_state; a.ckpt = p->checkpoints;
    a.status = p->status;
    return dispatch(a, p->x_dtype, p->g_dtype, kFwd, static_cast<cudaStream_t>(stream));
}

la_status glr_bwd(const la_glr_bwd_params* p, void* stream) {
    if (!p || p->D <= 0) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->g_dtype)) return LA_ERR_UNSUPPORTED;
    if (p->initial_state && !known_dtype(p->initial_state_dtype)) return LA_ERR_UNSUPPORTED;
    if ((st = check_gate(p->gate_mode, p->gate_lower_bound)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->g, p->g_stride_t, p->T, p->D, p->g_dtype, false) ||
        !good_rows(p->d_h, p->d_h_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->dx, p->dx_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_rows(p->dg, p->dg_stride_t, p->T, p->D, p->g_dtype, true) ||
        !good_optional(p->initial_state, p->initial_state_dtype) || !good_optional(p->checkpoints, LA_DTYPE_F32) ||
        !good_optional(p->d_final_state, LA_DTYPE_F32) || !good_optional(p->d_initial_state, LA_DTYPE_F32))
        return LA_ERR_INVALID_ARG;
    const size_t need = la_glr_workspace_bytes(p->T, p->N, p->D, 1, p->checkpoints != nullptr);
    if ((st = check_workspace(p->workspace, p->workspace_bytes, need)) != LA_OK) return st;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.g = p->g; a.g_st = p->g_stride_t;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D;
    a.mode = p->gate_mode; a.lb = p->gate_lower_bound; a.compl_in = p->complement_input != 0;
    a.s0 = p->initial_state; a.s0_bf16 = p->initial_state_dtype == LA_DTYPE_BF16;
    a.dh = p->d_h; a.dh_st = p->d_h_stride_t; a.dfin = p->d_final_state;
    a.dx = p->dx; a.dx_st = p->dx_stride_t; a.dg = p->dg; a.dg_st = p->dg_stride_t; a.ds0 = p->d_initial_state;
    a.status = p->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.ckpt = const_cast<float*>(p->checkpoints);
    if (!a.ckpt) {  // the forward again, for the states entering every block
        a.ckpt = static_cast<float*>(p->workspace);
        if ((st = dispatch(a, p->x_dtype, p->g_dtype, kFwd, s)) != LA_OK) return st;
    }
    return dispatch(a, p->x_dtype, p->g_dtype, kBwd, s);
}

la_status glr_decode(const la_glr_decode_params* p, void* stream) {
    if (!p || p->D <= 0 || p->N < 0) return LA_ERR_INVALID_ARG;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->g_dtype) || !known_dtype(p->state_dtype)) return LA_ERR_UNSUPPORTED;
    la_status st = check_gate(p->gate_mode, p->gate_lower_bound);
    if (st != LA_OK) return st;
    if (!p->state_pool || !good_optional(p->state_pool, p->state_dtype) || p->state_pool_size <= 0) return LA_ERR_INVALID_ARG;
    if (p->state_indices ? !aligned_to(p->state_indices, 4) : p->state_pool_size < p->N) return LA_ERR_INVALID_ARG;
    if (!good_rows(p->x, p->x_stride_n, p->N, p->D, p->x_dtype, false) ||
        !good_rows(p->g, p->g_stride_n, p->N, p->D, p->g_dtype, false) ||
        !good_rows(p->h, p->h_stride_n, p->N, p->D, p->x_dtype, true))
        return LA_ERR_INVALID_ARG;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_n; a.g = p->g; a.g_st = p->g_stride_n;
    a.N = p->N; a.D = p->D;
    a.mode = p->gate_mode; a.lb = p->gate_lower_bound; a.compl_in = p->complement_input != 0;
    a.s0 = p->state_pool; a.s0_bf16 = p->state_dtype == LA_DTYPE_BF16;
    a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.h = p->h; a.h_st = p->h_stride_n;
    a.status = p->status;
    return dispatch(a, p->x_dtype, p->g_dtype, kDecode, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
