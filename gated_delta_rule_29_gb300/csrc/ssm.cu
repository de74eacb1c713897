// ssm.cu -- the selective state space scan (ssm_fwd, ssm_bwd, ssm_decode): the single-token step and the entry points.
// The scans are in ssm_fwd.cu and ssm_bwd.cu, the formulas in ssm.cuh.
#include "ssm.cuh"

namespace {

using namespace la;
using namespace la::mixer;
using namespace la::ssm;

constexpr int kThreads = 128;

// One thread four states of one channel of one sequence.
template <typename X, int Q>
__global__ void __launch_bounds__(kThreads) ssm_decode_kernel(const Args a) {
    const int64_t i = this_slot();
    if (i >= a.N) return;
    const int q = threadIdx.x % Q, s = 4 * q;
    const int d = blockIdx.x * (kThreads / Q) + threadIdx.x / Q;
    const int64_t row = state_row(a, static_cast<int32_t>(i));
    if (row < 0) return;
    const bool live = d < a.D;
    const int j = live ? d / a.Dg : 0;
    float4 h = load_states(a.s0, row, a, d, s, live, a.s0_bf16);
    const float4 A = load_states(a.A, 0, a, d, s, live, 0);
    const float4 b = load4<X>(a.b, i * a.b_st + j * a.b_sg + s, a.S - s, a.vec), c = load4<X>(a.c, i * a.c_st + j * a.c_sg + s, a.S - s, a.vec);
    const float x = live ? to_f(static_cast<const X*>(a.x)[i * a.x_st + d]) : 0.f;
    const float dt = live ? steps_of(both(to_f(static_cast<const X*>(a.dt)[i * a.dt_st + d]) + (a.bias ? a.bias[d] : 0.f)), a.softplus).x : 0.f;
    const float u = dt * x, l = dt * kLog2e;
    h.x = fmaf(ex2(l * A.x), h.x, u * b.x);
    h.y = fmaf(ex2(l * A.y), h.y, u * b.y);
    h.z = fmaf(ex2(l * A.z), h.z, u * b.z);
    h.w = fmaf(ex2(l * A.w), h.w, u * b.w);
    store_states(const_cast<void*>(a.s0), row, a, d, s, live, a.s0_bf16, h);
    float p = fmaf(h.x, c.x, h.y * c.y) + fmaf(h.z, c.z, h.w * c.w);
#pragma unroll
    for (int off = 1; off < Q; off *= 2) p += __shfl_xor_sync(0xffffffffu, p, off);
    if (!live || q) return;
    if (a.skip) p = fmaf(a.skip[d], x, p);
    if (a.z) p *= act_fwd(LA_ACT_SILU, to_f(static_cast<const X*>(a.z)[i * a.z_st + d]));
    static_cast<X*>(a.y)[i * a.y_st + d] = from_f<X>(p);
}

struct Decode {
    template <typename X, int Q>
    static la_status run(Args& a, cudaStream_t s) {
        constexpr int kChannels = kThreads / Q;
        ssm_decode_kernel<X, Q><<<slot_grid((a.D + kChannels - 1) / kChannels, a.N), kThreads, 0, s>>>(a);
        return launched();
    }
};

template <typename X>
la_status by_states(Args& a, cudaStream_t s) {
    if (a.S <= 4) return Decode::run<X, 1>(a, s);
    if (a.S <= 8) return Decode::run<X, 2>(a, s);
    if (a.S <= 16) return Decode::run<X, 4>(a, s);
    if (a.S <= 32) return Decode::run<X, 8>(a, s);
    return Decode::run<X, 16>(a, s);
}

size_t round_up(size_t n) { return (n + 255) & ~size_t(255); }

bool good_shape(int32_t D, int32_t S, int32_t G) { return D > 0 && S > 0 && G > 0 && D % G == 0; }

// [rows, G, S] operands.
bool good_states(const void* p, int64_t st, int64_t sg, int64_t rows, int32_t dtype) {
    return rows == 0 || (p && aligned_to(p, dtype_size(dtype)) && st >= 0 && sg >= 0);
}

// Whether a result's rows lie over an operand's other than exactly over it, element by element.
bool clashes(const void* out, int64_t out_st, const void* in, int64_t in_st, int64_t rows, int64_t D, int32_t dtype) {
    if (!in || (out == in && (out_st == in_st || rows == 1))) return false;
    return rows_meet(out, out_st, in, in_st, rows, D, dtype);
}

template <typename P>
la_status check_common(const P* p, int64_t rows, int64_t x_st, int64_t dt_st, int64_t z_st, int64_t b_st, int64_t c_st) {
    if (!good_shape(p->D, p->S, p->G)) return LA_ERR_INVALID_ARG;
    if (p->S > kMaxS || !known_dtype(p->x_dtype)) return LA_ERR_UNSUPPORTED;
    if (!good_rows(p->x, x_st, rows, p->D, p->x_dtype, false) || !good_rows(p->dt, dt_st, rows, p->D, p->x_dtype, false) ||
        (p->z && !good_rows(p->z, z_st, rows, p->D, p->x_dtype, false)) || !good_states(p->b, b_st, p->b_stride_g, rows, p->x_dtype) ||
        !good_states(p->c, c_st, p->c_stride_g, rows, p->x_dtype))
        return LA_ERR_INVALID_ARG;
    if (!p->a || !aligned_to(p->a, 4) || !good_optional(p->skip, LA_DTYPE_F32) || !good_optional(p->dt_bias, LA_DTYPE_F32))
        return LA_ERR_INVALID_ARG;
    return LA_OK;
}

template <typename P>
void fill(Args& a, const P* p, int64_t rows, int64_t x_st, int64_t dt_st, int64_t z_st, int64_t b_st, int64_t c_st) {
    a.x = p->x; a.x_st = x_st; a.dt = p->dt; a.dt_st = dt_st; a.z = p->z; a.z_st = z_st;
    a.b = p->b; a.b_st = b_st; a.b_sg = p->b_stride_g; a.c = p->c; a.c_st = c_st; a.c_sg = p->c_stride_g;
    a.A = p->a; a.skip = p->skip; a.bias = p->dt_bias; a.softplus = p->dt_softplus != 0;
    a.N = p->N; a.T = rows; a.D = p->D; a.S = p->S; a.G = p->G; a.Dg = p->D / p->G;
    a.status = p->status;
    // rows whose channels, and states, start on 16-byte boundaries
    const int n = 16 / dtype_size(p->x_dtype);
    auto row = [&](const void* q, int64_t st) { return !q || (aligned_to(q, 16) && (rows <= 1 || st % n == 0)); };
    auto state = [&](const void* q, int64_t st, int64_t sg) { return row(q, st) && (a.G == 1 || sg % n == 0); };
    a.vec = row(p->x, x_st) && row(p->dt, dt_st) && row(p->z, z_st) && (a.G == 1 || a.Dg % n == 0) && state(p->b, b_st, p->b_stride_g) &&
            state(p->c, c_st, p->c_stride_g);
    a.svec = a.S % 4 == 0 && aligned_to(p->a, 16);
}
bool wide_rows(const Args& a, const void* p, int64_t st, int32_t dtype) {
    return !p || (aligned_to(p, 16) && (a.T <= 1 || st % (16 / dtype_size(dtype)) == 0));
}

template <typename P>
void fill_seqs(Args& a, const P* p) {
    a.cu = p->cu_seqlens; a.cu64 = p->cu_seqlens_bits == 64;
    a.s0 = p->initial_state; a.s0_bf16 = p->initial_state_dtype == LA_DTYPE_BF16;
    a.svec = a.svec && aligned_to(p->initial_state, 16);
}

bool good_time_block(int32_t b) { return b == 0 || (b >= 64 && (b & (b - 1)) == 0 && b <= (1 << 30)); }

// The forward's workspace: what enters each time block, and the steps' sums; nothing where no sequence can have two.
size_t table_bytes(int64_t T, int32_t N, int32_t D, int32_t S, int shift) {
    if (!split(T, shift)) return 0;
    const size_t slots = static_cast<size_t>(slots_for(T, N, shift));
    return round_up(slots * D * S * 4) + round_up(slots * D * 4);
}
void set_table(Args& a, void* ws, int shift) {
    a.table = static_cast<float*>(ws);
    a.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round_up(static_cast<size_t>(slots_for(a.T, a.N, shift)) * a.D * a.S * 4));
}

}  // namespace

extern "C" {

size_t la_ssm_checkpoint_rows(int64_t T, int32_t N) {
    return T < 0 || N < 0 ? 0 : static_cast<size_t>(T / kSave + N);
}

size_t la_ssm_fwd_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t S, int32_t G, int32_t time_block) {
    if (T < 0 || N < 0 || !good_shape(D, S, G) || S > kMaxS || !good_time_block(time_block)) return 0;
    return table_bytes(T, N, D, S, fwd_shift(T, D, S, G, time_block));
}

size_t la_ssm_bwd_workspace_bytes(int64_t T, int32_t N, int32_t D, int32_t S, int32_t G, int32_t checkpoints_given) {
    if (T < 0 || N < 0 || !good_shape(D, S, G) || S > kMaxS) return 0;
    const size_t DS = static_cast<size_t>(D) * S, rows = la_ssm_checkpoint_rows(T, N), parts = bwd_parts(T, N, D, S, G), blocks = bwd_blocks(T, N);
    const size_t tiles = (D / G + bwd_width(S) - 1) / bwd_width(S);
    size_t n = round_up(blocks * DS * 4) + round_up(blocks * D * 4) + round_up(tiles * T * G * 2 * S * 4) + round_up(parts * DS * 4) +
               round_up(parts * 2 * D * 4);
    if (!checkpoints_given) n += round_up(rows * DS * 4) + la_ssm_fwd_workspace_bytes(T, N, D, S, G, 0);
    return n;
}

la_status ssm_fwd(const la_ssm_fwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if ((st = check_common(p, p->T, p->x_stride_t, p->dt_stride_t, p->z_stride_t, p->b_stride_t, p->c_stride_t)) != LA_OK) return st;
    if (p->initial_state && !known_dtype(p->initial_state_dtype)) return LA_ERR_UNSUPPORTED;
    if (!good_rows(p->y, p->y_stride_t, p->T, p->D, p->x_dtype, true) || !good_optional(p->initial_state, p->initial_state_dtype) ||
        !good_optional(p->final_state, LA_DTYPE_F32) || !good_optional(p->checkpoints, LA_DTYPE_F32) || !good_time_block(p->time_block))
        return LA_ERR_INVALID_ARG;
    if (clashes(p->y, p->y_stride_t, p->x, p->x_stride_t, p->T, p->D, p->x_dtype) || clashes(p->y, p->y_stride_t, p->dt, p->dt_stride_t, p->T, p->D, p->x_dtype) ||
        clashes(p->y, p->y_stride_t, p->z, p->z_stride_t, p->T, p->D, p->x_dtype))
        return LA_ERR_INVALID_ARG;
    if (p->state_indices && (!aligned_to(p->state_indices, 4) || !p->initial_state || p->final_state || p->state_pool_size <= 0))
        return LA_ERR_INVALID_ARG;
    Args a = {};
    fill(a, p, p->T, p->x_stride_t, p->dt_stride_t, p->z_stride_t, p->b_stride_t, p->c_stride_t);
    fill_seqs(a, p);
    a.shift = fwd_shift(a.T, a.D, a.S, a.G, p->time_block);
    if ((st = check_workspace(p->workspace, p->workspace_bytes, table_bytes(a.T, a.N, a.D, a.S, a.shift))) != LA_OK) return st;
    set_table(a, p->workspace, a.shift);
    a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.y = p->y; a.y_st = p->y_stride_t; a.fin = p->final_state; a.ckpt = p->checkpoints;
    a.vec = a.vec && wide_rows(a, a.y, a.y_st, p->x_dtype);
    a.svec = a.svec && aligned_to(a.fin, 16) && aligned_to(a.ckpt, 16);
    if (a.N == 0) return LA_OK;
    return run_fwd(a, p->x_dtype, static_cast<cudaStream_t>(stream));
}

la_status ssm_bwd(const la_ssm_bwd_params* p, void* stream) {
    if (!p) return LA_ERR_INVALID_ARG;
    la_status st = check_seqs(p->cu_seqlens, p->cu_seqlens_bits, p->N, p->T);
    if (st != LA_OK) return st;
    if ((st = check_common(p, p->T, p->x_stride_t, p->dt_stride_t, p->z_stride_t, p->b_stride_t, p->c_stride_t)) != LA_OK) return st;
    if (p->initial_state && !known_dtype(p->initial_state_dtype)) return LA_ERR_UNSUPPORTED;
    const int32_t xd = p->x_dtype;
    if (!good_rows(p->dy, p->dy_stride_t, p->T, p->D, xd, false) || !good_rows(p->dx, p->dx_stride_t, p->T, p->D, xd, true) ||
        !good_rows(p->ddt, p->ddt_stride_t, p->T, p->D, xd, true) || (p->z && !good_rows(p->dz, p->dz_stride_t, p->T, p->D, xd, true)) ||
        !good_states(p->db, 0, 0, p->T, xd) || !good_states(p->dc, 0, 0, p->T, xd))
        return LA_ERR_INVALID_ARG;
    if (!p->da || !aligned_to(p->da, 4) || (p->skip && !p->d_skip) || (p->dt_bias && !p->d_dt_bias) || !good_optional(p->d_skip, LA_DTYPE_F32) ||
        !good_optional(p->d_dt_bias, LA_DTYPE_F32) || !good_optional(p->initial_state, p->initial_state_dtype) ||
        !good_optional(p->checkpoints, LA_DTYPE_F32) || !good_optional(p->d_final_state, LA_DTYPE_F32) ||
        !good_optional(p->d_initial_state, LA_DTYPE_F32))
        return LA_ERR_INVALID_ARG;
    const size_t need = la_ssm_bwd_workspace_bytes(p->T, p->N, p->D, p->S, p->G, p->checkpoints != nullptr);
    if ((st = check_workspace(p->workspace, p->workspace_bytes, need)) != LA_OK) return st;
    Args a = {};
    fill(a, p, p->T, p->x_stride_t, p->dt_stride_t, p->z_stride_t, p->b_stride_t, p->c_stride_t);
    fill_seqs(a, p);
    a.dy = p->dy; a.dy_st = p->dy_stride_t;
    a.dx = p->dx; a.dx_st = p->dx_stride_t; a.ddt = p->ddt; a.ddt_st = p->ddt_stride_t; a.dz = p->dz; a.dz_st = p->dz_stride_t;
    a.db = p->db; a.dc = p->dc; a.dA = p->da; a.dskip = p->skip ? p->d_skip : nullptr; a.dbias = p->dt_bias ? p->d_dt_bias : nullptr;
    a.dfin = p->d_final_state; a.ds0 = p->d_initial_state;
    a.vec = a.vec && wide_rows(a, a.dy, a.dy_st, xd) && wide_rows(a, a.dx, a.dx_st, xd) && wide_rows(a, a.ddt, a.ddt_st, xd) &&
            wide_rows(a, a.dz, a.dz_st, xd);
    a.svec = a.svec && aligned_to(p->checkpoints, 16);
    a.parts = bwd_parts(a.T, a.N, a.D, a.S, a.G);
    const size_t DS = static_cast<size_t>(a.D) * a.S, rows = la_ssm_checkpoint_rows(a.T, a.N), blocks = bwd_blocks(a.T, a.N);
    const size_t tiles = (a.Dg + bwd_width(a.S) - 1) / bwd_width(a.S);
    uint8_t* ws = static_cast<uint8_t*>(p->workspace);
    auto take = [&](size_t bytes) {
        float* q = reinterpret_cast<float*>(ws);
        ws += round_up(bytes);
        return q;
    };
    float* table = take(blocks * DS * 4);
    float* sums = take(blocks * a.D * 4);
    a.dbc = take(tiles * a.T * a.G * 2 * a.S * 4);
    a.pA = take(static_cast<size_t>(a.parts) * DS * 4);
    a.pch = take(static_cast<size_t>(a.parts) * 2 * a.D * 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.ckpt = const_cast<float*>(p->checkpoints);
    if (!a.ckpt && a.N > 0) {  // the forward again, for the states entering every chunk
        a.ckpt = take(rows * DS * 4);
        Args f = a;
        f.shift = fwd_shift(a.T, a.D, a.S, a.G, 0);
        set_table(f, ws, f.shift);
        f.y = nullptr;
        if ((st = run_fwd(f, xd, s)) != LA_OK) return st;
    }
    a.table = table;
    a.sums = sums;
    return run_bwd(a, xd, s);
}

la_status ssm_decode(const la_ssm_decode_params* p, void* stream) {
    if (!p || p->N < 0) return LA_ERR_INVALID_ARG;
    la_status st = check_common(p, p->N, p->x_stride_n, p->dt_stride_n, p->z_stride_n, p->b_stride_n, p->c_stride_n);
    if (st != LA_OK) return st;
    if (!known_dtype(p->state_dtype)) return LA_ERR_UNSUPPORTED;
    if (!p->state_pool || !good_optional(p->state_pool, p->state_dtype) || p->state_pool_size <= 0) return LA_ERR_INVALID_ARG;
    if (p->state_indices ? !aligned_to(p->state_indices, 4) : p->state_pool_size < p->N) return LA_ERR_INVALID_ARG;
    if (!good_rows(p->y, p->y_stride_n, p->N, p->D, p->x_dtype, true)) return LA_ERR_INVALID_ARG;
    Args a = {};
    fill(a, p, p->N, p->x_stride_n, p->dt_stride_n, p->z_stride_n, p->b_stride_n, p->c_stride_n);
    a.s0 = p->state_pool; a.s0_bf16 = p->state_dtype == LA_DTYPE_BF16;
    a.svec = a.svec && aligned_to(a.s0, 16);
    a.idx = p->state_indices; a.pool = p->state_pool_size;
    a.y = p->y; a.y_st = p->y_stride_n;
    if (a.N == 0) return LA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return p->x_dtype == LA_DTYPE_BF16 ? by_states<bf16>(a, s) : by_states<float>(a, s);
}

}  // extern "C"
