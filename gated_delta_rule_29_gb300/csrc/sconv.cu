// sconv.cu -- the short causal convolution with an activation (sconv_fwd, sconv_bwd, sconv_decode).
//
// Per channel of each sequence, x_s for s < 0 being the initial state's rows:
//
//   p_t = b + sum_j w_j x_{t - (W - 1) + j},  y_t = act(p_t);
//   dp_t = dy_t act'(p_t),  dx_t = sum_j w_j dp_{t + (W - 1) - j} (+ the final state's gradient),
//   dw_j = sum_t dp_t x_{t - (W - 1) + j},  db = sum_t dp_t.
//
// A thread walks kSpan consecutive tokens of its channels with the W - 1 tokens before them in
// registers; the eight warps of a CTA take the eight spans of a 128-token block.  The backward
// recomputes p, looks W - 1 tokens past its span, and leaves one partial sum of dw and db per
// block, which a second kernel adds in order.
#include <algorithm>

#include "mixer.cuh"

namespace {

using namespace la::mixer;

constexpr int kThreads = 256;
constexpr int kBlock = 128;
constexpr int kSpan = kBlock / (kThreads / 32);

struct Args {
    const void *x, *w, *b, *cu, *s0, *dy, *dfin;
    int64_t x_st, y_st, dy_st, dx_st, T;
    int cu64, N, D, w_bf16, act;
    const int32_t* idx;
    int64_t pool;
    void *y, *fin, *dx, *ds0;
    float* part;  // [slots][W + 1][D]: dw_0 .. dw_{W-1}, db
    int32_t* status;
};

// Input of channel d at place pos of the sequence that starts at `first`: a token, or a row of the
// state before it.
template <typename X, int W>
__device__ __forceinline__ float input_at(const Args& a, int64_t first, int64_t slot, int64_t pos, int d) {
    if (pos >= 0) return to_f(static_cast<const X*>(a.x)[(first + pos) * a.x_st + d]);
    return a.s0 ? to_f(static_cast<const X*>(a.s0)[(slot * (W - 1) + (W - 1) + pos) * a.D + d]) : 0.f;
}

// The state slot of sequence i, or false when its index is outside the pool.
__device__ __forceinline__ bool state_slot(const Args& a, int i, int64_t& slot) {
    slot = i;
    if (!a.idx) return true;
    slot = a.idx[i];
    if (slot >= 0 && slot < a.pool) return true;
    raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
    return false;
}

template <typename X, int W>
__global__ void __launch_bounds__(kThreads) sconv_fwd_kernel(const Args a) {
    const int64_t slot_id = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
    const int d = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
    if (slot_id >= a.T / kBlock + a.N) return;
    if (blockIdx.x == 0)
        for (int64_t i = slot_id * kThreads + threadIdx.x; i < a.N && i < (slot_id + 1) * kThreads; i += kThreads)
            check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
    const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, slot_id);
    int64_t slot;
    if (b.seq < 0 || d >= a.D || !state_slot(a, b.seq, slot)) return;
    float w[W], win[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = load_any(a.w, static_cast<int64_t>(d) * W + j, a.w_bf16);
    const float bias = a.b ? load_any(a.b, d, a.w_bf16) : 0.f;
    const int k0 = warp * kSpan, k1 = min(k0 + kSpan, b.count);
    const int64_t p0 = static_cast<int64_t>(b.c) * kBlock;
    if (k0 < k1) {
#pragma unroll
        for (int j = 1; j < W; ++j) win[j] = input_at<X, W>(a, b.first, slot, p0 + k0 - W + j, d);
        for (int k = k0; k < k1; ++k) {
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1];
            win[W - 1] = input_at<X, W>(a, b.first, slot, p0 + k, d);
            float p = bias;
#pragma unroll
            for (int j = 0; j < W; ++j) p = fmaf(w[j], win[j], p);
            static_cast<X*>(a.y)[(static_cast<int64_t>(b.start) + k) * a.y_st + d] = from_f<X>(act_fwd(a.act, p));
        }
    }
    // The sequence's last W - 1 inputs.  With a pool they replace the rows that the sequence started
    // from, which only this thread reads: they reach the first W - 1 tokens, and kSpan is no less.
    if (b.c == 0 && warp == 0 && (a.fin || a.idx)) {
        float f[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) f[j] = input_at<X, W>(a, b.first, slot, b.len - (W - 1) + j, d);
        X* to = a.idx ? static_cast<X*>(const_cast<void*>(a.s0)) + slot * (W - 1) * a.D
                      : static_cast<X*>(a.fin) + static_cast<int64_t>(b.seq) * (W - 1) * a.D;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) to[static_cast<int64_t>(j) * a.D + d] = from_f<X>(f[j]);
    }
}

// dp of the token at place pos (0 beyond the sequence's end).
template <typename X, int W>
__device__ __forceinline__ float dp_at(const Args& a, const SeqBlock& b, const float (&w)[W], const float (&win)[W],
                                       float bias, int64_t pos, int d) {
    if (pos < 0 || pos >= b.len) return 0.f;
    float p = bias, g;
#pragma unroll
    for (int j = 0; j < W; ++j) p = fmaf(w[j], win[j], p);
    act_grad(a.act, p, g);
    return g * to_f(static_cast<const X*>(a.dy)[(b.first + pos) * a.dy_st + d]);
}

template <typename X, int W>
__global__ void __launch_bounds__(kThreads) sconv_bwd_kernel(const Args a) {
    __shared__ float red[kThreads / 32][W + 1][32];
    const int64_t slot_id = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
    const int lane = threadIdx.x & 31, d = blockIdx.x * 32 + lane, warp = threadIdx.x >> 5;
    if (slot_id >= a.T / kBlock + a.N) return;
    if (blockIdx.x == 0)
        for (int64_t i = slot_id * kThreads + threadIdx.x; i < a.N && i < (slot_id + 1) * kThreads; i += kThreads)
            check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
    const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, slot_id);
    float dw[W], db = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = 0.f;
    const int k0 = warp * kSpan, k1 = min(k0 + kSpan, b.count);
    const int64_t p0 = static_cast<int64_t>(b.c) * kBlock;
    if (b.seq >= 0 && d < a.D && k0 < k1) {
        float w[W], win[W], dp[W];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = load_any(a.w, static_cast<int64_t>(d) * W + j, a.w_bf16);
        const float bias = a.b ? load_any(a.b, d, a.w_bf16) : 0.f;
        // dp[j]: dp of place k + j, the window of the place W - 1 further on being in win
#pragma unroll
        for (int j = 1; j < W; ++j) win[j] = input_at<X, W>(a, b.first, b.seq, p0 + k0 - W + j, d);
#pragma unroll
        for (int k = 0; k < kSpan + W - 1; ++k) {
            const int64_t pos = p0 + k0 + k;
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) {
                win[j] = win[j + 1];
                dp[j] = k == 0 ? 0.f : dp[j + 1];
            }
            win[W - 1] = pos < b.len ? input_at<X, W>(a, b.first, b.seq, pos, d) : 0.f;
            dp[W - 1] = dp_at<X, W>(a, b, w, win, bias, pos, d);
            if (k < kSpan && pos < b.len) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j] = fmaf(dp[W - 1], win[j], dw[j]);
                db += dp[W - 1];
            }
            if (k >= W - 1 && k0 + k - (W - 1) < k1) {
                const int64_t at = pos - (W - 1);
                float dx = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) dx = fmaf(w[j], dp[W - 1 - j], dx);
                const int64_t f = at - (b.len - (W - 1));
                if (a.dfin && f >= 0) dx += to_f(static_cast<const X*>(a.dfin)[(b.seq * int64_t(W - 1) + f) * a.D + d]);
                static_cast<X*>(a.dx)[(b.first + at) * a.dx_st + d] = from_f<X>(dx);
            }
        }
    }
    // d(initial state): the rows before the first token, through the tokens they reach
    if (b.seq >= 0 && b.c == 0 && a.ds0 && d < a.D && warp == 0) {
        float w[W], dp[W - 1];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = load_any(a.w, static_cast<int64_t>(d) * W + j, a.w_bf16);
        const float bias = a.b ? load_any(a.b, d, a.w_bf16) : 0.f;
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            float win[W];
#pragma unroll
            for (int j = 0; j < W; ++j) win[j] = t < b.len && t - (W - 1) + j < b.len
                                                     ? input_at<X, W>(a, b.first, b.seq, t - (W - 1) + j, d) : 0.f;
            dp[t] = dp_at<X, W>(a, b, w, win, bias, t, d);
        }
#pragma unroll
        for (int s = 0; s < W - 1; ++s) {  // the row at place s - (W - 1) is tap s - t of token t <= s
            float ds = 0.f;
#pragma unroll
            for (int t = 0; t <= s; ++t) ds = fmaf(w[s - t], dp[t], ds);
            const int64_t f = s - b.len;
            if (a.dfin && f >= 0) ds += to_f(static_cast<const X*>(a.dfin)[(b.seq * int64_t(W - 1) + f) * a.D + d]);
            static_cast<X*>(a.ds0)[(b.seq * int64_t(W - 1) + s) * a.D + d] = from_f<X>(ds);
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) red[warp][j][lane] = dw[j];
    red[warp][W][lane] = db;
    __syncthreads();
    if (warp <= W && d < a.D) {
        float s = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) s += red[i][warp][lane];
        a.part[(slot_id * (W + 1) + warp) * a.D + d] = s;
    }
}

// dw[d][j] and db[d]: the partial sums of all slots.  A CTA takes 32 channels of one j; its warps take
// every eighth slot, in order.
template <int W>
__global__ void __launch_bounds__(256) sconv_sum_kernel(const float* part, int64_t slots, int D, void* dw, void* db,
                                                        int w_bf16) {
    __shared__ float sh[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.y;
    const int d = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (d < D)
        for (int64_t k = warp; k < slots; k += 8) s += part[(k * (W + 1) + j) * D + d];
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < D) {
        for (int i = 1; i < 8; ++i) s += sh[i][lane];
        if (j < W) store_any(dw, static_cast<int64_t>(d) * W + j, w_bf16, s);
        else if (db) store_any(db, d, w_bf16, s);
    }
}

template <typename X, int W>
__global__ void __launch_bounds__(kThreads) sconv_decode_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = blockIdx.x * kThreads + threadIdx.x;
    int64_t slot;
    if (i >= a.N || d >= a.D || !state_slot(a, i, slot)) return;
    X* st = static_cast<X*>(const_cast<void*>(a.s0)) + slot * (W - 1) * a.D + d;
    float win[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = to_f(st[static_cast<int64_t>(j) * a.D]);
    win[W - 1] = to_f(static_cast<const X*>(a.x)[i * a.x_st + d]);
    float p = a.b ? load_any(a.b, d, a.w_bf16) : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) p = fmaf(load_any(a.w, static_cast<int64_t>(d) * W + j, a.w_bf16), win[j], p);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) st[static_cast<int64_t>(j) * a.D] = from_f<X>(win[j + 1]);
    static_cast<X*>(a.y)[i * a.y_st + d] = from_f<X>(act_fwd(a.act, p));
}

enum Which { kFwd, kBwd, kDecode };

template <typename X, int W>
la_status launch(const Args& a, Which w, cudaStream_t s) {
    const int64_t blocks = w == kDecode ? a.N : a.T / kBlock + a.N;
    if (blocks == 0) return LA_OK;
    const int64_t ny = std::min<int64_t>(blocks, 65535), nz = (blocks + ny - 1) / ny;
    const dim3 grid((a.D + (w == kDecode ? kThreads : 32) - 1) / (w == kDecode ? kThreads : 32),
                    static_cast<unsigned>(ny), static_cast<unsigned>(nz));
    if (w == kFwd) sconv_fwd_kernel<X, W><<<grid, kThreads, 0, s>>>(a);
    else if (w == kBwd) sconv_bwd_kernel<X, W><<<grid, kThreads, 0, s>>>(a);
    else sconv_decode_kernel<X, W><<<grid, kThreads, 0, s>>>(a);
    return launched();
}

template <typename X>
la_status dispatch_w(const Args& a, int W, Which w, cudaStream_t s) {
    if (W == 2) return launch<X, 2>(a, w, s);
    if (W == 3) return launch<X, 3>(a, w, s);
    return launch<X, 4>(a, w, s);
}

la_status dispatch(const Args& a, int W, int32_t xd, Which w, cudaStream_t s) {
    return xd == LA_DTYPE_BF16 ? dispatch_w<bf16>(a, W, w, s) : dispatch_w<float>(a, W, w, s);
}

la_status check(int32_t D, int32_t W, int32_t xd, int32_t wd, int32_t act, const void* w, const void* b) {
    if (D <= 0) return LA_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || !known_dtype(xd) || !known_dtype(wd)) return LA_ERR_UNSUPPORTED;
    if (act < LA_ACT_NONE || act > LA_ACT_SIGMOID) return LA_ERR_INVALID_ARG;
    if (!w || !aligned_to(w, dtype_size(wd)) || !good_optional(b, wd)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

}  // namespace

extern "C" {

size_t la_sconv_bwd_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t W) {
    if (T < 0 || N < 0 || D <= 0 || W < 2 || W > 4) return 0;
    return (static_cast<size_t>(T / kBlock + N) * (W + 1) * D * 4 + 255) & ~size_t(255);
}

la_status sconv_fwd(const la_sconv_fwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if ((st = check(p->D, p->W, p->x_dtype, p->weight_dtype, p->activation, p->weight, p->bias)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->y, p->y_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_optional(p->initial_state, p->x_dtype) || !good_optional(p->final_state, p->x_dtype))
        return LA_ERR_INVALID_ARG;
    if (p->state_indices && (!aligned_to(p->state_indices, 4) || !p->initial_state || p->final_state || p->state_pool_size <= 0))
        return LA_ERR_INVALID_ARG;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D; a.act = p->activation;
    a.s0 = p->initial_state; a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.y = p->y; a.y_st = p->y_stride_t; a.fin = p->final_state; a.status = p->status;
    return dispatch(a, p->W, p->x_dtype, kFwd, static_cast<cudaStream_t>(stream));
}

la_status sconv_bwd(const la_sconv_bwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if ((st = check(p->D, p->W, p->x_dtype, p->weight_dtype, p->activation, p->weight, p->bias)) != LA_OK) return st;
    if (!good_rows(p->x, p->x_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->dy, p->dy_stride_t, p->T, p->D, p->x_dtype, false) ||
        !good_rows(p->dx, p->dx_stride_t, p->T, p->D, p->x_dtype, true) ||
        !good_optional(p->initial_state, p->x_dtype) || !good_optional(p->d_final_state, p->x_dtype) ||
        !good_optional(p->d_initial_state, p->x_dtype))
        return LA_ERR_INVALID_ARG;
    if (!p->d_weight || !aligned_to(p->d_weight, dtype_size(p->weight_dtype)) || (p->bias && !p->d_bias) ||
        !good_optional(p->d_bias, p->weight_dtype))
        return LA_ERR_INVALID_ARG;
    if ((st = check_workspace(p->workspace, p->workspace_bytes, la_sconv_bwd_workspace_bytes(p->T, p->N, p->D, p->W))) != LA_OK)
        return st;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_t; a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64; a.T = p->T; a.N = p->N; a.D = p->D; a.act = p->activation;
    a.s0 = p->initial_state; a.dy = p->dy; a.dy_st = p->dy_stride_t; a.dfin = p->d_final_state;
    a.dx = p->dx; a.dx_st = p->dx_stride_t; a.ds0 = p->d_initial_state;
    a.part = static_cast<float*>(p->workspace); a.status = p->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = dispatch(a, p->W, p->x_dtype, kBwd, s)) != LA_OK) return st;
    const dim3 grid((a.D + 31) / 32, p->W + (p->bias ? 1 : 0));
    const int64_t slots = a.T / kBlock + a.N;
    void* db = p->bias ? p->d_bias : nullptr;
    if (p->W == 2) sconv_sum_kernel<2><<<grid, 256, 0, s>>>(a.part, slots, a.D, p->d_weight, db, a.w_bf16);
    else if (p->W == 3) sconv_sum_kernel<3><<<grid, 256, 0, s>>>(a.part, slots, a.D, p->d_weight, db, a.w_bf16);
    else sconv_sum_kernel<4><<<grid, 256, 0, s>>>(a.part, slots, a.D, p->d_weight, db, a.w_bf16);
    return launched();
}

la_status sconv_decode(const la_sconv_decode_params* p, void* stream) {
    if (!p || p->N < 0) return LA_ERR_INVALID_ARG;
    la_status st = check(p->D, p->W, p->x_dtype, p->weight_dtype, p->activation, p->weight, p->bias);
    if (st != LA_OK) return st;
    if (!p->state_pool || !good_optional(p->state_pool, p->x_dtype) || p->state_pool_size <= 0) return LA_ERR_INVALID_ARG;
    if (p->state_indices ? !aligned_to(p->state_indices, 4) : p->state_pool_size < p->N) return LA_ERR_INVALID_ARG;
    if (!good_rows(p->x, p->x_stride_n, p->N, p->D, p->x_dtype, false) ||
        !good_rows(p->y, p->y_stride_n, p->N, p->D, p->x_dtype, true))
        return LA_ERR_INVALID_ARG;
    Args a = {};
    a.x = p->x; a.x_st = p->x_stride_n; a.w = p->weight; a.b = p->bias; a.w_bf16 = p->weight_dtype == LA_DTYPE_BF16;
    a.N = p->N; a.D = p->D; a.act = p->activation;
    a.s0 = p->state_pool; a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.y = p->y; a.y_st = p->y_stride_n; a.status = p->status;
    return dispatch(a, p->W, p->x_dtype, kDecode, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
