// ssm.cu -- the selective state space scan (ssm_fwd, ssm_bwd, ssm_decode): the single-token step and the entry points.
// The scans are in ssm_fwd.cu and ssm_bwd.cu, the formulas in ssm.cuh.
#include "ssm.cuh"

namespace {

using namespace la;
using namespace la::mixer;
using namespace la::ssm;

constexpr int kThreads = 128;

// The two kernels below sum C h in one order, (h0 c0 + h2 c2) + (h1 c1 + h3 c3) of every four states and then pairs of fours, pairs
// of those and so on, so that a sequence's bits do not depend on how many others are decoded beside it.

// A lane has kS states of one channel of one sequence: as few steps are formed as there are channels, but its 16-byte
// accesses lie kS * 4 bytes from its neighbours' (512 x 8192 x 16 in fp32: 124 us, all of it L1 wavefronts).
// Into a bf16 pool (kBf16) the new states are formed by the formula's own operations, each rounded once, with the library's
// exponential and logarithm: an error of some 2^-24 puts one in 10^5 states on the other side of a rounding to 8 bits, half a
// percent away, and the tokens after it see that.  512 x 8192 x 16 into such a pool: 105 us, 337 with accesses of single states.
template <typename X, int kS, int Q, bool kBf16>
__global__ void __launch_bounds__(kThreads) ssm_decode_kernel(const Args a) {
    constexpr int kW = 32 / Q, kPairs = kS / 2;  // channels of a warp
    const int lane = threadIdx.x & 31, q = lane / kW, s0 = kS * q;
    const int d = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kW + lane % kW;
    const int64_t i = this_slot();
    if (i >= a.N) return;
    const bool live = d < a.D;
    const int64_t row = state_row(a, static_cast<int32_t>(i));
    if (row < 0) return;
    float2 h[kPairs], A[kPairs];
    load_lane_states<kS>(h, a.s0, row, a, d, s0, live, kBf16);
    const float x = live ? to_f(static_cast<const X*>(a.x)[i * a.x_st + d]) : 0.f, raw = live ? to_f(static_cast<const X*>(a.dt)[i * a.dt_st + d]) : 0.f;
    const float z = live && a.z ? to_f(static_cast<const X*>(a.z)[i * a.z_st + d]) : 0.f;
    load_lane_states<kS>(A, a.A, 0, a, d, s0, live, 0);
    const float bias = live && a.bias ? a.bias[d] : 0.f, skip = live && a.skip ? a.skip[d] : 0.f;
    const int64_t j = live ? d / a.Dg : 0, b_at = i * a.b_st + j * a.b_sg + s0, c_at = i * a.c_st + j * a.c_sg + s0;
    float step;
    if (kBf16 && a.softplus) step = __fadd_rn(fmaxf(raw + bias, 0.f), log1pf(expf(-fabsf(raw + bias))));
    else step = steps_of(both(raw + bias), a.softplus).x;
    const float2 u = both(__fmul_rn(step, x));
    auto next = [&](float2& h, float2 A, float2 b) {
        if (kBf16) {
            h.x = __fadd_rn(__fmul_rn(expf(__fmul_rn(step, A.x)), h.x), __fmul_rn(u.x, b.x));
            h.y = __fadd_rn(__fmul_rn(expf(__fmul_rn(step, A.y)), h.y), __fmul_rn(u.x, b.y));
        } else {
            const float2 e = fma2(both(step), mul2(A, both(kLog2e)), both(kEx2Low));
            h = fma2(make_float2(ex2(e.x), ex2(e.y)), h, mul2(u, b));
        }
    };
    float y[kS / 4];
#pragma unroll
    for (int k = 0; k < kPairs; k += 2) {
        const float4 b = load4<X>(a.b, b_at + 2 * k, a.S - s0 - 2 * k, a.vec), c = load4<X>(a.c, c_at + 2 * k, a.S - s0 - 2 * k, a.vec);
        next(h[k], A[k], lo(b));
        next(h[k + 1], A[k + 1], hi(b));
        const float2 t = fma2(h[k], lo(c), mul2(h[k + 1], hi(c)));
        y[k / 2] = t.x + t.y;
    }
    store_lane_states<kS>(h, const_cast<void*>(a.s0), row, a, d, s0, live, kBf16);
#pragma unroll
    for (int n = 1; n < kS / 4; n *= 2)
#pragma unroll
        for (int k = 0; k < kS / 4; k += 2 * n) y[k] += y[k + n];
    float p = y[0];
#pragma unroll
    for (int off = kW; off < 32; off *= 2) p += __shfl_xor_sync(0xffffffffu, p, off);
    p = fmaf(skip, x, p);
    if (a.z) p *= act_fwd(LA_ACT_SILU, z);
    if (live && q == 0) static_cast<X*>(a.y)[i * a.y_st + d] = from_f<X>(p);
}

// For many fp32 states: Q neighbouring lanes share a channel, four states each, so that accesses are contiguous, and a CTA
// keeps its channels and goes over the sequences, four at a time, with the states of the next groups on their way into shared
// memory (each thread's own 16 bytes, so that nothing waits but the thread).  The lanes of a channel share the four
// sequences' steps and results.  512 x 8192 x 16 in 112 us (4.8 TB/s), 512 x 4096 x 64 in 219 (375 the way above).
constexpr int kSeqs = 4, kDepth = 4;

template <typename X, int Q>
__global__ void __launch_bounds__(kThreads, 4) ssm_decode_many_kernel(const Args a, int64_t groups) {
    __shared__ __align__(16) float4 ring[kDepth][kSeqs][kThreads];
    constexpr int kShare = Q < kSeqs ? Q : kSeqs, kOwn = kSeqs / kShare;  // lanes that share the sequences; sequences of a lane
    const int q = threadIdx.x % Q, s = 4 * q, mine = q % kShare;          // this lane's: mine, mine + kShare, ...
    const int d = blockIdx.x * (kThreads / Q) + threadIdx.x / Q;
    const bool live = d < a.D && s < a.S;
    const int dl = min(d, a.D - 1), j = dl / a.Dg;
    const int64_t within = static_cast<int64_t>(dl) * a.S + s, pitch = static_cast<int64_t>(a.D) * a.S;
    float* const pool = static_cast<float*>(const_cast<void*>(a.s0));
    const float bias = a.bias ? a.bias[dl] : 0.f, skip = a.skip ? a.skip[dl] : 0.f;
    float4 A = load_states(a.A, 0, a, d, s, live, 0);  // times log2(e)
    A = make_float4(A.x * kLog2e, A.y * kLog2e, A.z * kLog2e, A.w * kLog2e);

    // the slots of a group's sequences as they are given; which of them are there is seen when they are used
    auto slots_of = [&](int (&slot)[kSeqs], int64_t group) {
#pragma unroll
        for (int i = 0; i < kSeqs; ++i) {
            const int64_t n = group * kSeqs + i;
            slot[i] = n < a.N ? (a.idx ? a.idx[n] : static_cast<int>(n)) : -1;
        }
    };
    auto request = [&](int stage, const int (&slot)[kSeqs]) {
#pragma unroll
        for (int i = 0; i < kSeqs; ++i)
            if (live && slot[i] >= 0 && slot[i] < a.pool) cp_async16(&ring[stage][i][threadIdx.x], pool + slot[i] * pitch + within);
        cp_async_commit();
    };
    struct Inputs {
        Packed<X, 4> b[kSeqs], c[kSeqs];
        X x[kOwn], dt[kOwn], z[kOwn];
    };
    auto inputs_of = [&](int64_t group) {
        Inputs t;
#pragma unroll
        for (int i = 0; i < kSeqs; ++i) {
            const int64_t n = min(group * kSeqs + i, int64_t(a.N) - 1);
            t.b[i].load(static_cast<const X*>(a.b) + n * a.b_st + j * a.b_sg + min(s, a.S - 4));
            t.c[i].load(static_cast<const X*>(a.c) + n * a.c_st + j * a.c_sg + min(s, a.S - 4));
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int64_t n = min(group * kSeqs + mine + k * kShare, int64_t(a.N) - 1);
            t.x[k] = static_cast<const X*>(a.x)[n * a.x_st + dl];
            t.dt[k] = static_cast<const X*>(a.dt)[n * a.dt_st + dl];
            t.z[k] = a.z ? static_cast<const X*>(a.z)[n * a.z_st + dl] : from_f<X>(0.f);
        }
        return t;
    };
    const int64_t step = gridDim.y;
    int64_t group = blockIdx.y;
    int slot[kDepth][kSeqs];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) slots_of(slot[k], group + k * step);
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) request(k, slot[k]);
    Inputs in = inputs_of(group);
    for (int64_t n = 0; group < groups; ++n, group += step) {
        request(static_cast<int>((n + kDepth - 1) % kDepth), slot[kDepth - 1]);
        int here[kSeqs];
#pragma unroll
        for (int i = 0; i < kSeqs; ++i) {
            here[i] = slot[0][i];
#pragma unroll
            for (int k = 0; k + 1 < kDepth; ++k) slot[k][i] = slot[k + 1][i];
        }
        slots_of(slot[kDepth - 1], group + kDepth * step);
        const Inputs now = in;
        in = inputs_of(group + step);
        float x[kOwn], dt[kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            x[k] = to_f(now.x[k]);
            dt[k] = steps_of(both(to_f(now.dt[k]) + bias), a.softplus).x;
        }
        cp_async_wait<kDepth - 1>();
        float p[kSeqs];
#pragma unroll
        for (int i = 0; i < kSeqs; ++i) {
            const int from = (threadIdx.x & 31) / Q * Q + i % kShare;
            const float t = kShare == 1 ? dt[i / kShare] : __shfl_sync(0xffffffffu, dt[i / kShare], from);
            const float v = kShare == 1 ? x[i / kShare] : __shfl_sync(0xffffffffu, x[i / kShare], from);
            const bool there = here[i] >= 0 && here[i] < a.pool;
            const float u = t * v;
            float4 h = ring[n % kDepth][i][threadIdx.x];
            h.x = fmaf(ex2(fmaf(t, A.x, kEx2Low)), h.x, u * now.b[i].get(0));
            h.y = fmaf(ex2(fmaf(t, A.y, kEx2Low)), h.y, u * now.b[i].get(1));
            h.z = fmaf(ex2(fmaf(t, A.z, kEx2Low)), h.z, u * now.b[i].get(2));
            h.w = fmaf(ex2(fmaf(t, A.w, kEx2Low)), h.w, u * now.b[i].get(3));
            if (live && there) *reinterpret_cast<float4*>(pool + here[i] * pitch + within) = h;
            p[i] = live ? fmaf(h.x, now.c[i].get(0), h.z * now.c[i].get(2)) + fmaf(h.y, now.c[i].get(1), h.w * now.c[i].get(3)) : 0.f;
            if (Q == 1) p[i] += 0.f;  // the other kernel's four states beyond: -0 becomes 0
#pragma unroll
            for (int off = 1; off < Q; off *= 2) p[i] += __shfl_xor_sync(0xffffffffu, p[i], off);
            if (!there && group * kSeqs + i < a.N) raise_status(a.status, LA_ERR_BAD_STATE_INDEX);
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            float y = 0.f;
            bool there = false;
#pragma unroll
            for (int i = 0; i < kShare; ++i)
                if (mine == i) {
                    y = p[i + k * kShare];
                    there = here[i + k * kShare] >= 0 && here[i + k * kShare] < a.pool;
                }
            y = fmaf(skip, x[k], y);
            if (a.z) y *= act_fwd(LA_ACT_SILU, to_f(now.z[k]));
            if (there && d < a.D && q < kShare) static_cast<X*>(a.y)[(group * kSeqs + mine + k * kShare) * a.y_st + d] = from_f<X>(y);
        }
    }
    cp_async_wait<0>();
}

template <typename X, int kS, int Q>
la_status decode(const Args& a, cudaStream_t s) {
    constexpr int kChannels = kThreads / Q;
    const dim3 grid = slot_grid((a.D + kChannels - 1) / kChannels, a.N);
    if (a.s0_bf16) ssm_decode_kernel<X, kS, Q, true><<<grid, kThreads, 0, s>>>(a);
    else ssm_decode_kernel<X, kS, Q, false><<<grid, kThreads, 0, s>>>(a);
    return launched();
}
template <typename X, int Q>
la_status decode_many(const Args& a, cudaStream_t s) {
    const int tiles = (a.D + kThreads / Q - 1) / (kThreads / Q);
    const int64_t groups = (int64_t(a.N) + kSeqs - 1) / kSeqs;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(std::min<int64_t>(65535, std::max<int64_t>(1, groups / 8))));
    ssm_decode_many_kernel<X, Q><<<grid, kThreads, 0, s>>>(a, groups);
    return launched();
}
template <typename X>
la_status by_states(const Args& a, cudaStream_t s) {
    // rows in 16-byte accesses throughout, and states enough for CTAs of eight groups: 64 x 8192 x 16 takes 21 us this way and
    // 25 the other, 64 x 4096 x 16 18 and 16
    if (a.vec && a.svec && !a.s0_bf16 && a.S >= 4 && static_cast<int64_t>(a.N) * a.D * a.S >= int64_t(1) << 23) {
        if (a.S <= 4) return decode_many<X, 1>(a, s);
        if (a.S <= 8) return decode_many<X, 2>(a, s);
        if (a.S <= 16) return decode_many<X, 4>(a, s);
        if (a.S <= 32) return decode_many<X, 8>(a, s);
        return decode_many<X, 16>(a, s);
    }
    if (a.S <= 8) return decode<X, 8, 1>(a, s);
    if (a.S <= 16) return decode<X, 16, 1>(a, s);
    if (a.S <= 32) return decode<X, 16, 2>(a, s);
    return decode<X, 16, 4>(a, s);
}

size_t round_up(size_t n) { return (n + 255) & ~size_t(255); }

bool good_shape(int32_t D, int32_t S, int32_t G) { return D > 0 && S > 0 && G > 0 && D % G == 0; }

// [rows, G, S] operands.
bool good_states(const void* p, int64_t st, int64_t sg, int64_t rows, int32_t dtype) {
    return rows == 0 || (p && aligned_to(p, dtype_size(dtype)) && st >= 0 && sg >= 0);
}

// Whether rows of D elements share memory with b's or c's vectors, which every channel of a group reads.
template <typename P>
bool over_vectors(const P* p, const void* rows_at, int64_t st, int64_t rows, int64_t b_st, int64_t c_st) {
    const int64_t es = dtype_size(p->x_dtype);
    auto over = [&](const void* v, int64_t v_st, int64_t v_sg) {
        if (!bytes_meet(rows_at, st * es, p->D * es, v, v_st * es, ((p->G - 1) * v_sg + p->S) * es, rows)) return false;
        for (int64_t j = 0; j < (v_sg ? p->G : 1); ++j)
            if (bytes_meet(rows_at, st * es, p->D * es, static_cast<const uint8_t*>(v) + j * v_sg * es, v_st * es, p->S * es, rows)) return true;
        return false;
    };
    return rows_at && (over(p->b, b_st, p->b_stride_g) || over(p->c, c_st, p->c_stride_g));
}

// Whether y shares memory with x, dt or z other than by lying exactly over one of them, or with b or c.
template <typename P>
bool result_clashes(const P* p, int64_t rows, int64_t y_st, int64_t x_st, int64_t dt_st, int64_t z_st, int64_t b_st, int64_t c_st) {
    const int64_t es = dtype_size(p->x_dtype);
    auto over = [&](const void* in, int64_t st) { return clashes(p->y, y_st, es, in, st, es, rows, p->D); };
    return over(p->x, x_st) || over(p->dt, dt_st) || over(p->z, z_st) || over_vectors(p, p->y, y_st, rows, b_st, c_st);
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
    if (result_clashes(p, p->T, p->y_stride_t, p->x_stride_t, p->dt_stride_t, p->z_stride_t, p->b_stride_t, p->c_stride_t)) return LA_ERR_INVALID_ARG;
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
    // no gradient may lie over an input, which other warps still read, or over another gradient
    const struct {
        const void* p;
        int64_t st;
    } rows_of[] = {{p->dx, p->dx_stride_t}, {p->ddt, p->ddt_stride_t}, {p->z ? p->dz : nullptr, p->dz_stride_t}, {p->x, p->x_stride_t},
                   {p->dt, p->dt_stride_t}, {p->dy, p->dy_stride_t}, {p->z, p->z_stride_t}};
    for (int i = 0; i < 3; ++i) {
        if (over_vectors(p, rows_of[i].p, rows_of[i].st, p->T, p->b_stride_t, p->c_stride_t)) return LA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 7; ++j)
            if (rows_of[i].p && rows_of[j].p && rows_meet(rows_of[i].p, rows_of[i].st, rows_of[j].p, rows_of[j].st, p->T, p->D, xd))
                return LA_ERR_INVALID_ARG;
    }
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
        f.z = nullptr;
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
    if (!good_rows(p->y, p->y_stride_n, p->N, p->D, p->x_dtype, true) ||
        result_clashes(p, p->N, p->y_stride_n, p->x_stride_n, p->dt_stride_n, p->z_stride_n, p->b_stride_n, p->c_stride_n))
        return LA_ERR_INVALID_ARG;
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
