// sconv.cu -- the short causal convolution with an activation (sconv_fwd, sconv_bwd, sconv_decode).
//
// Per channel of each sequence, x_s for s < 0 being the initial state's rows:
//
//   p_t = b + sum_j w_j x_{t - (W - 1) + j},  y_t = act(p_t);
//   dp_t = dy_t act'(p_t),  dx_t = sum_j w_j dp_{t + (W - 1) - j} (+ the final state's gradient),
//   dw_j = sum_t dp_t x_{t - (W - 1) + j},  db = sum_t dp_t.
//
// A thread walks 16 consecutive tokens of its channels (four, where rows allow 4-element accesses) with
// the W - 1 tokens before them in registers; the eight warps of a CTA take the eight spans of a 128-token
// block.  A span's loads are issued in groups ahead of its arithmetic.  The backward recomputes p, looks
// W - 1 tokens past its span, and leaves one partial sum of dw and db per block (20 bytes a channel for
// 128 tokens at W = 4), which a second kernel adds in order.
#include <algorithm>

#include "mixer.cuh"

namespace {

using namespace la::mixer;

constexpr int kThreads = 256, kDecodeThreads = 128;
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

// The state slot of sequence i, or false when its index is outside the pool.
__device__ __forceinline__ bool state_slot(const Args& a, int i, int64_t& slot) {
    slot = i;
    if (!a.idx) return true;
    slot = a.idx[i];
    if (slot >= 0 && slot < a.pool) return true;
    raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
    return false;
}

// The input at place pos < 0 or < len of a sequence: a token, or a row of the state before it.
template <typename X, int kVec, int W>
__device__ __forceinline__ void input_at(Packed<X, kVec>& v, const Args& a, int64_t first, int64_t slot, int64_t pos, int d) {
    if (pos >= 0) v.load(static_cast<const X*>(a.x) + (first + pos) * a.x_st + d);
    else if (a.s0) v.load(static_cast<const X*>(a.s0) + (slot * (W - 1) + (W - 1) + pos) * a.D + d);
    else v.zero();
}

template <int kVec, int W>
__device__ __forceinline__ void load_taps(float (&w)[W][kVec], float (&bias)[kVec], const Args& a, int d) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = load_any(a.w, static_cast<int64_t>(d + i) * W + j, a.w_bf16);
        bias[i] = a.b ? load_any(a.b, d + i, a.w_bf16) : 0.f;
    }
}

__device__ __forceinline__ void check_boundaries(const Args& a, int64_t slot) {
    if (blockIdx.x == 0)
        for (int64_t i = slot * kThreads + threadIdx.x; i < a.N && i < (slot + 1) * kThreads; i += kThreads)
            check_cu(a.cu, a.cu64, a.N, a.T, i, a.status);
}

template <typename X, int W, int kVec>
__global__ void __launch_bounds__(kThreads) sconv_fwd_kernel(const Args a) {
    constexpr int kGroup = 8;  // tokens whose loads are issued together
    const int64_t slot_id = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
    const int d = (blockIdx.x * 32 + (threadIdx.x & 31)) * kVec, warp = threadIdx.x >> 5;
    if (slot_id >= a.T / kBlock + a.N) return;
    check_boundaries(a, slot_id);
    const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, slot_id);
    int64_t slot;
    if (b.seq < 0 || d >= a.D || !state_slot(a, b.seq, slot)) return;
    const int k0 = warp * kSpan, n = min(kSpan, b.count - k0);
    const int64_t p0 = static_cast<int64_t>(b.c) * kBlock + k0;
    if (n > 0) {
        float w[W][kVec], bias[kVec], win[W][kVec];
        Packed<X, kVec> raw[kGroup];
        Packed<X, kVec> before[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<X, kVec, W>(before[j], a, b.first, slot, p0 - (W - 1) + j, d);
        const X* px = static_cast<const X*>(a.x) + (static_cast<int64_t>(b.start) + k0) * a.x_st + d;
        X* py = static_cast<X*>(a.y) + (static_cast<int64_t>(b.start) + k0) * a.y_st + d;
        load_taps<kVec, W>(w, bias, a, d);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) win[j + 1][i] = before[j].get(i);
#pragma unroll
        for (int g = 0; g < kSpan; g += kGroup) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
                if (g + k < n) raw[k].load(px + (g + k) * a.x_st);
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
                if (g + k < n) {
                    float y[kVec];
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
#pragma unroll
                        for (int j = 0; j + 1 < W; ++j) win[j][i] = win[j + 1][i];
                        win[W - 1][i] = raw[k].get(i);
                        float p = bias[i];
#pragma unroll
                        for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                        y[i] = act_fwd(a.act, p);
                    }
                    store_packed<X, kVec>(py + (g + k) * a.y_st, y);
                }
        }
    }
    // The sequence's last W - 1 inputs.  With a pool they replace the rows that the sequence started
    // from, which only this thread reads: they reach the first W - 1 tokens, and kSpan is no less.
    if (b.c == 0 && warp == 0 && (a.fin || a.idx)) {
        Packed<X, kVec> f[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<X, kVec, W>(f[j], a, b.first, slot, static_cast<int64_t>(b.len) - (W - 1) + j, d);
        X* to = a.idx ? static_cast<X*>(const_cast<void*>(a.s0)) + slot * (W - 1) * a.D
                      : static_cast<X*>(a.fin) + static_cast<int64_t>(b.seq) * (W - 1) * a.D;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float v[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] = f[j].get(i);
            store_packed<X, kVec>(to + static_cast<int64_t>(j) * a.D + d, v);
        }
    }
}

template <typename X, int W, int kVec>
__global__ void __launch_bounds__(kThreads) sconv_bwd_kernel(const Args a) {
    constexpr int kGroup = 4, kSteps = (kSpan + W - 1 + kGroup - 1) / kGroup * kGroup;
    __shared__ float red[kThreads / 32][W + 1][32 * kVec];
    const int64_t slot_id = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
    const int lane = threadIdx.x & 31, d = (blockIdx.x * 32 + lane) * kVec, warp = threadIdx.x >> 5;
    if (slot_id >= a.T / kBlock + a.N) return;
    check_boundaries(a, slot_id);
    const SeqBlock b = find_block<kBlock>(a.cu, a.cu64, a.N, a.T, slot_id);
    const bool mine = b.seq >= 0 && d < a.D;
    float dw[W][kVec] = {}, db[kVec] = {};
    const int k0 = warp * kSpan, n = min(kSpan, b.count - k0);
    const int64_t p0 = static_cast<int64_t>(b.c) * kBlock + k0;
    if (mine && n > 0) {
        float w[W][kVec], bias[kVec], win[W][kVec], dp[W][kVec];
        Packed<X, kVec> before[W - 1], raw[kGroup], raw_dy[kGroup];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<X, kVec, W>(before[j], a, b.first, b.seq, p0 - (W - 1) + j, d);
        load_taps<kVec, W>(w, bias, a, d);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j + 1][i] = before[j].get(i);
#pragma unroll
            for (int j = 0; j < W; ++j) dp[j][i] = 0.f;
        }
        const int64_t t0 = static_cast<int64_t>(b.start) + k0;
        const X* px = static_cast<const X*>(a.x) + t0 * a.x_st + d;
        const X* pdy = static_cast<const X*>(a.dy) + t0 * a.dy_st + d;
        X* pdx = static_cast<X*>(a.dx) + t0 * a.dx_st + d;
        const int left = static_cast<int>(min(b.len - p0, static_cast<int64_t>(kSteps)));  // tokens from here to the sequence's end
#pragma unroll
        for (int g = 0; g < kSteps; g += kGroup) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                if (g + k < kSpan + W - 1 && g + k < left) {
                    raw[k].load(px + (g + k) * a.x_st);
                    raw_dy[k].load(pdy + (g + k) * a.dy_st);
                } else {  // beyond the end: dp = 0
                    raw[k].zero();
                    raw_dy[k].zero();
                }
            }
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int at = g + k;  // the token whose dp this step forms; dx follows W - 1 tokens behind
                if (at >= kSpan + W - 1) continue;
                float dx[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) {
                        win[j][i] = win[j + 1][i];
                        dp[j][i] = dp[j + 1][i];
                    }
                    win[W - 1][i] = raw[k].get(i);
                    float p = bias[i], slope;
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                    act_grad(a.act, p, slope);
                    const float v = at < left ? raw_dy[k].get(i) * slope : 0.f;
                    dp[W - 1][i] = v;
                    if (at < kSpan) {
                        if (at < left) {
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][i] = fmaf(v, win[j][i], dw[j][i]);
                            db[i] += v;
                        }
                    }
                    dx[i] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) dx[i] = fmaf(w[j][i], dp[W - 1 - j][i], dx[i]);
                }
                const int out = at - (W - 1);
                if (out >= 0 && out < n) {
                    const int64_t f = p0 + out - (static_cast<int64_t>(b.len) - (W - 1));
                    if (a.dfin && f >= 0) {
                        Packed<X, kVec> e;
                        e.load(static_cast<const X*>(a.dfin) + (b.seq * static_cast<int64_t>(W - 1) + f) * a.D + d);
#pragma unroll
                        for (int i = 0; i < kVec; ++i) dx[i] += e.get(i);
                    }
                    store_packed<X, kVec>(pdx + out * a.dx_st, dx);
                }
            }
        }
    }
    // d(initial state): the rows before the first token, through the tokens they reach
    if (mine && b.c == 0 && a.ds0 && warp == 0) {
        float w[W][kVec], bias[kVec], dp[W - 1][kVec];
        load_taps<kVec, W>(w, bias, a, d);
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            Packed<X, kVec> in[W], dy;
            dy.zero();
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (t < b.len) input_at<X, kVec, W>(in[j], a, b.first, b.seq, t - (W - 1) + j, d);
                else in[j].zero();
            }
            if (t < b.len) dy.load(static_cast<const X*>(a.dy) + (static_cast<int64_t>(b.first) + t) * a.dy_st + d);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                float p = bias[i], slope;
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][i], in[j].get(i), p);
                act_grad(a.act, p, slope);
                dp[t][i] = t < b.len ? slope * dy.get(i) : 0.f;
            }
        }
#pragma unroll
        for (int s = 0; s < W - 1; ++s) {  // the row at place s - (W - 1) is tap s - t of token t <= s
            float ds[kVec];
            Packed<X, kVec> e;
            e.zero();
            const int f = s - b.len;
            if (a.dfin && f >= 0) e.load(static_cast<const X*>(a.dfin) + (b.seq * static_cast<int64_t>(W - 1) + f) * a.D + d);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                ds[i] = e.get(i);
#pragma unroll
                for (int t = 0; t <= s; ++t) ds[i] = fmaf(w[s - t][i], dp[t][i], ds[i]);
            }
            store_packed<X, kVec>(static_cast<X*>(a.ds0) + (b.seq * static_cast<int64_t>(W - 1) + s) * a.D + d, ds);
        }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[warp][j][lane * kVec + i] = dw[j][i];
        red[warp][W][lane * kVec + i] = db[i];
    }
    __syncthreads();
    const int width = min(32 * kVec, a.D - static_cast<int>(blockIdx.x) * 32 * kVec);
    for (int e = threadIdx.x; e < (W + 1) * 32 * kVec; e += kThreads) {
        const int j = e / (32 * kVec), c = e % (32 * kVec);
        if (c >= width) continue;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) s += red[i][j][c];
        a.part[(slot_id * (W + 1) + j) * a.D + blockIdx.x * 32 * kVec + c] = s;
    }
}

// dw[d][j] and db[d]: the partial sums of all slots.  A CTA takes 32 channels of one j; its 32 warps take
// every 32nd slot, in order.
template <int W>
__global__ void __launch_bounds__(1024) sconv_sum_kernel(const float* part, int64_t slots, int D, void* dw, void* db,
                                                         int w_bf16) {
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.y;
    const int d = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (d < D) {
#pragma unroll 8
        for (int64_t k = warp; k < slots; k += 32) s += part[(k * (W + 1) + j) * D + d];
    }
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sh[i][lane];
        if (j < W) store_any(dw, static_cast<int64_t>(d) * W + j, w_bf16, s);
        else if (db) store_any(db, d, w_bf16, s);
    }
}

template <typename X, int W, int kVec>
__global__ void __launch_bounds__(kDecodeThreads) sconv_decode_kernel(const Args a) {
    const int i = blockIdx.y + gridDim.y * blockIdx.z;
    const int d = (blockIdx.x * kDecodeThreads + threadIdx.x) * kVec;
    int64_t slot;
    if (i >= a.N || d >= a.D || !state_slot(a, i, slot)) return;
    X* st = static_cast<X*>(const_cast<void*>(a.s0)) + slot * (W - 1) * a.D + d;
    Packed<X, kVec> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j].load(st + static_cast<int64_t>(j) * a.D);
    in[W - 1].load(static_cast<const X*>(a.x) + i * a.x_st + d);
    float w[W][kVec], bias[kVec], y[kVec];
    load_taps<kVec, W>(w, bias, a, d);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        float p = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(w[j][e], in[j].get(e), p);
        y[e] = act_fwd(a.act, p);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float v[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = in[j + 1].get(e);
        store_packed<X, kVec>(st + static_cast<int64_t>(j) * a.D, v);
    }
    store_packed<X, kVec>(static_cast<X*>(a.y) + i * a.y_st + d, y);
}

enum Which { kFwd, kBwd, kDecode };

template <typename X, int W, int kVec>
la_status launch(const Args& a, Which w, cudaStream_t s) {
    const int64_t blocks = w == kDecode ? a.N : a.T / kBlock + a.N;
    if (blocks == 0) return LA_OK;
    const int64_t ny = std::min<int64_t>(blocks, 65535), nz = (blocks + ny - 1) / ny;
    const int width = (w == kDecode ? kDecodeThreads : 32) * kVec;
    const dim3 grid((a.D + width - 1) / width, static_cast<unsigned>(ny), static_cast<unsigned>(nz));
    if (w == kFwd) sconv_fwd_kernel<X, W, kVec><<<grid, kThreads, 0, s>>>(a);
    else if (w == kBwd) sconv_bwd_kernel<X, W, kVec><<<grid, kThreads, 0, s>>>(a);
    else sconv_decode_kernel<X, W, kVec><<<grid, kDecodeThreads, 0, s>>>(a);
    return launched();
}

// Four channels a lane where every operand's rows start on four of its elements.
template <typename X, int W>
la_status by_vec(const Args& a, Which w, cudaStream_t s) {
    const int bytes = 4 * static_cast<int>(sizeof(X));
    auto ok = [&](const void* p, int64_t st) { return !p || (aligned_to(p, bytes) && st % 4 == 0); };
    const bool four = a.D % 4 == 0 && ok(a.x, a.x_st) && ok(a.y, a.y_st) && ok(a.dy, a.dy_st) && ok(a.dx, a.dx_st) && ok(a.s0, 0) &&
                      ok(a.fin, 0) && ok(a.dfin, 0) && ok(a.ds0, 0);
    return four ? launch<X, W, 4>(a, w, s) : launch<X, W, 1>(a, w, s);
}

template <typename X>
la_status dispatch_w(const Args& a, int W, Which w, cudaStream_t s) {
    if (W == 2) return by_vec<X, 2>(a, w, s);
    if (W == 3) return by_vec<X, 3>(a, w, s);
    return by_vec<X, 4>(a, w, s);
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
    if (p->W == 2) sconv_sum_kernel<2><<<grid, 1024, 0, s>>>(a.part, slots, a.D, p->d_weight, db, a.w_bf16);
    else if (p->W == 3) sconv_sum_kernel<3><<<grid, 1024, 0, s>>>(a.part, slots, a.D, p->d_weight, db, a.w_bf16);
    else sconv_sum_kernel<4><<<grid, 1024, 0, s>>>(a.part, slots, a.D, p->d_weight, db, a.w_bf16);
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
