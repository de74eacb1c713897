// glr.cu -- the gated linear recurrence (glr_fwd, glr_bwd, glr_decode): the single-token step and the entry points.
// The scans are in glr_fwd.cu and glr_bwd.cu, the method in glr.cuh.
#include "glr.cuh"

namespace {

using namespace la;
using namespace la::mixer;
using namespace la::glr;

constexpr int kThreads = 128;

// One thread a channel: a step of 8 x 2048 takes 4 us on the GPU, all latency (state index, then state), and the call
// 12 us of host time.
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
    float dec, m;
    const float g = to_f(static_cast<const G*>(a.g)[i * a.g_st + d]);
    with_gate(a.mode, a.compl_in, [&](auto gt) {
        const Gated t = gate<decltype(gt)::mode, decltype(gt)::complement>(a.lb, both(g));
        dec = t.a.x;
        m = t.m.x;
    });
    const float h = fmaf(dec, load_any(a.s0, slot * a.D + d, a.s0_bf16), m * to_f(static_cast<const X*>(a.x)[i * a.x_st + d]));
    store_any(const_cast<void*>(a.s0), slot * a.D + d, a.s0_bf16, h);
    static_cast<X*>(a.h)[i * a.h_st + d] = from_f<X>(h);
}

// The chain's table: maps and states of every item.  None when no sequence can have two blocks.
size_t map_bytes(int64_t T, int32_t N, int32_t D) {
    if (T <= kBlock) return 0;
    return static_cast<size_t>(T / kBlock + N) * ((D + kChannels - 1) / kChannels) * 32 * sizeof(ulonglong2);
}
size_t table_bytes(int64_t T, int32_t N, int32_t D) { return map_bytes(T, N, D) / 2 * 3; }  // a state is half a map

enum Which { kFwd, kBwd };

la_status run_scan(Args& a, int32_t xd, int32_t gd, Which w, void* ws, cudaStream_t s) {
    if (a.N == 0) return LA_OK;
    a.tiles = (a.D + kChannels - 1) / kChannels;
    a.items = (a.T / kBlock + a.N) * a.tiles;
    if (a.items >= (int64_t(1) << 31)) return LA_ERR_UNSUPPORTED;
    if (const size_t maps = map_bytes(a.T, a.N, a.D)) {
        a.maps = static_cast<ulonglong2*>(ws);
        a.states = reinterpret_cast<uint2*>(static_cast<uint8_t*>(ws) + maps);
        if (cudaMemsetAsync(ws, 0xFF, table_bytes(a.T, a.N, a.D), s) != cudaSuccess) return LA_ERR_CUDA;
    }
    return w == kFwd ? run_fwd(a, xd, gd, s) : run_bwd(a, xd, gd, s);
}

template <typename X, typename G>
la_status launch_decode(const Args& a, cudaStream_t s) {
    const unsigned ny = std::min(a.N, 65535), nz = (a.N + ny - 1) / ny;
    glr_decode_kernel<X, G><<<dim3((a.D + kThreads - 1) / kThreads, ny, nz), kThreads, 0, s>>>(a);
    return launched();
}

}  // namespace

extern "C" {

size_t la_glr_checkpoint_rows(int64_t T, int32_t N) {
    return T < 0 || N < 0 ? 0 : static_cast<size_t>(T / kBlock + N);
}

size_t la_glr_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t backward, int32_t checkpoints_given) {
    if (T < 0 || N < 0 || D <= 0) return 0;
    const size_t states = backward && !checkpoints_given ? (la_glr_checkpoint_rows(T, N) * D * 4 + 255) & ~size_t(255) : 0;
    return states + table_bytes(T, N, D);
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
    return run_scan(a, p->x_dtype, p->g_dtype, kFwd, p->workspace, static_cast<cudaStream_t>(stream));
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
    if (!a.ckpt && a.N > 0) {  // the forward again, for the states entering every block, which come after the table
        Args f = a;
        f.ckpt = a.ckpt = reinterpret_cast<float*>(static_cast<uint8_t*>(p->workspace) + table_bytes(a.T, a.N, a.D));
        if ((st = run_scan(f, p->x_dtype, p->g_dtype, kFwd, p->workspace, s)) != LA_OK) return st;
    }
    return run_scan(a, p->x_dtype, p->g_dtype, kBwd, p->workspace, s);
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
    if (a.N == 0) return LA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->x_dtype == LA_DTYPE_BF16) return p->g_dtype == LA_DTYPE_BF16 ? launch_decode<bf16, bf16>(a, s) : launch_decode<bf16, float>(a, s);
    return p->g_dtype == LA_DTYPE_BF16 ? launch_decode<float, bf16>(a, s) : launch_decode<float, float>(a, s);
}

}  // extern "C"
