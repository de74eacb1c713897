// mixer.cuh -- what the token-mixer operators (glr, gn, sconv) and those of a state-space block (ssm, rn) share: element
// access in bf16 or fp32, activations, the numbering of sequence blocks, and host-side argument checks.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/liblinattn.h"
#include "ptx.cuh"
#include "seq_search.h"

namespace la {
namespace mixer {

typedef __nv_bfloat16 bf16;

// ---------------------------------------------------------------- element access
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }

// An element of a bf16 or fp32 array whose type is known at run time (parameters, states).
__device__ __forceinline__ float load_any(const void* p, int64_t i, int is_bf16) {
    return is_bf16 ? to_f(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int64_t i, int is_bf16, float x) {
    if (is_bf16) static_cast<bf16*>(p)[i] = from_f<bf16>(x);
    else static_cast<float*>(p)[i] = x;
}

// kVec consecutive elements as one access of kVec * sizeof(T) <= 16 bytes (aligned to that).
template <typename T, int kVec>
struct Packed {
    static constexpr int kWords = (kVec * static_cast<int>(sizeof(T)) + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) {
        if (kVec * sizeof(T) == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
        else if (kVec * sizeof(T) == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        else if (kVec * sizeof(T) == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
        else w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};
template <typename T, int kVec>
__device__ __forceinline__ void store_packed(T* p, const float (&v)[kVec]) {
    if (sizeof(T) == 4) {
        if (kVec == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[kVec > 1 ? 1 : 0], v[kVec > 2 ? 2 : 0], v[kVec > 3 ? 3 : 0]);
        else if (kVec == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[kVec > 1 ? 1 : 0]);
        else
#pragma unroll
            for (int i = 0; i < kVec; ++i) p[i] = from_f<T>(v[i]);
    } else if (kVec == 1) {
        p[0] = from_f<T>(v[0]);
    } else {
        uint32_t w[kVec / 2 > 0 ? kVec / 2 : 1];
#pragma unroll
        for (int i = 0; i + 1 < kVec; i += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[i], v[i + 1]);
            w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if (kVec == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[kVec > 2 ? 1 : 0], w[kVec > 4 ? 2 : 0], w[kVec > 6 ? 3 : 0]);
        else if (kVec == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[kVec > 2 ? 1 : 0]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// ---------------------------------------------------------------- two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tadd.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// ---------------------------------------------------------------- exponentials and activations
// e^l is ex2(l kLog2e): the product's rounding is off by |l| 2^-24 of the result, which is small where the result is
// not; results below 2^-126 are zero.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-x); e^-x may overflow to infinity, which gives the right 0.
__device__ __forceinline__ float sigmoidf(float x) { return rcp_fast(1.f + ex2(-x * kLog2e)); }

__device__ __forceinline__ float act_fwd(int kind, float p) {
    if (kind == LA_ACT_NONE) return p;
    const float s = sigmoidf(p);
    return kind == LA_ACT_SIGMOID ? s : p * s;
}
// The same for two values at once, and act' beside it, s being the sigmoid: silu' = s (1 + p (1 - s)), sigmoid' = s (1 - s).
template <int kAct>
__device__ __forceinline__ float2 act_fwd2(float2 p) {
    if (kAct == LA_ACT_NONE) return p;
    const float2 t = mul2(p, both(-kLog2e));
    const float2 q = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.f)), s = make_float2(rcp_fast(q.x), rcp_fast(q.y));
    return kAct == LA_ACT_SIGMOID ? s : mul2(p, s);
}
template <int kAct>
__device__ __forceinline__ float2 act_grad2(float2 p, float2& d) {
    if (kAct == LA_ACT_NONE) {
        d = both(1.f);
        return p;
    }
    if (kAct == LA_ACT_SIGMOID) {
        // 1 - s is e^-p s: a difference would lose its bits as s nears 1, and the derivative with them.  Beyond 2^126,
        // where s is 0, e^-p is held finite, so that the derivative is 0.
        const float2 t = mul2(p, both(-kLog2e)), e = make_float2(ex2(t.x), ex2(t.y)), q = add2(e, both(1.f));
        const float2 s = make_float2(rcp_fast(q.x), rcp_fast(q.y));
        d = mul2(s, mul2(make_float2(fminf(e.x, 0x1p126f), fminf(e.y, 0x1p126f)), s));
        return s;
    }
    // here the difference, off by 2^-23 at most, stands beside 1: an error of |p| 2^-23, no more than the exponential's
    // (49344 x 2048 backward through the convolution 133 us; 141 with the product)
    const float2 s = act_fwd2<LA_ACT_SIGMOID>(p), rest = fma2(s, both(-1.f), both(1.f));
    d = mul2(s, fma2(p, rest, both(1.f)));
    return mul2(p, s);
}

// p[first pitch] + p[(first + step) pitch] + ... below row `rows`, in order, kGroup loads at a time.
template <int kGroup>
__device__ __forceinline__ float strided_sum(const float* p, int64_t pitch, int64_t first, int64_t rows, int64_t step) {
    float s = 0.f;
    for (int64_t r = first; r < rows; r += kGroup * step) {
        float v[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) v[i] = r + i * step < rows ? p[(r + i * step) * pitch] : 0.f;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) s += v[i];
    }
    return s;
}

// ---------------------------------------------------------------- sequence blocks
__device__ __forceinline__ int64_t cu_load(const void* cu, int cu64, int64_t i) {
    return cu64 ? static_cast<const int64_t*>(cu)[i] : static_cast<int64_t>(static_cast<const int32_t*>(cu)[i]);
}

__device__ __forceinline__ void raise_status(int32_t* status, int32_t code) {
    if (status) atomicCAS(status, LA_OK, code);
}

// The block in `slot`; called by whole warps.  32-ary search over cu[i] / B + i, one round of loads
// for up to 32 sequences, two for up to 1024.  With invalid cu_seqlens the answer is some block
// inside [0, T), so that no access leaves the operands, and `same` says whether the same search for the
// slot `beside` ends at the same sequence (as it does where boundaries are valid and the sequence has a
// block there).
template <int B>
__device__ __forceinline__ SeqBlock find_block(const void* cu, int cu64, int32_t N, int64_t T, int64_t slot, int64_t beside, bool& same) {
    const int lane = threadIdx.x & 31;
    SlotSearch f = {0, N, true};
    while (f.n > 1) {
        const int32_t i = f.lo + lane * f.step();
        const bool live = lane * f.step() < f.n;
        const int64_t v = live ? cu_load(cu, cu64, i) / B + i : 0;
        const unsigned here = __ballot_sync(0xffffffffu, live && v <= slot);
        f.narrow(here, beside == slot ? here : __ballot_sync(0xffffffffu, live && v <= beside));
    }
    same = f.same;
    return block_of<B>(f.lo, cu_load(cu, cu64, f.lo), cu_load(cu, cu64, f.lo + 1), T, slot);
}
template <int B>
__device__ __forceinline__ SeqBlock find_block(const void* cu, int cu64, int32_t N, int64_t T, int64_t slot) {
    bool same;
    return find_block<B>(cu, cu64, N, T, slot, slot, same);
}

// Checks entry i of cu_seqlens (0 <= i < N, with its right neighbour and the two ends).
__device__ __forceinline__ void check_cu(const void* cu, int cu64, int32_t N, int64_t T, int64_t i, int32_t* status) {
    const int64_t a = cu_load(cu, cu64, i), b = cu_load(cu, cu64, i + 1);
    if (a < 0 || b < a || b > T || (i == 0 && a != 0) || (i == N - 1 && b != T)) raise_status(status, LA_ERR_BAD_SEQLENS);
}

// ---------------------------------------------------------------- tiles of a [T, D] operand by TMA
__device__ __forceinline__ void tile_load(void* dst, const CUtensorMap* map, uint64_t* bar, int channel, int token) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(channel), "r"(token), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tile_store(const CUtensorMap* map, const void* src, int channel, int token) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(channel),
                 "r"(token), "r"(smem_u32(src))
                 : "memory");
}

// Tiles of `rows` tokens x `channels` channels of a [T, D] operand, rows packed in shared memory.
inline bool tile_map(CUtensorMap* m, const void* p, int64_t stride, int64_t T, int64_t D, int32_t dtype, int channels, int rows) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Encode>(f) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t es = dtype == LA_DTYPE_BF16 ? 2 : 4;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(T == 1 ? (D * es + 15) / 16 * 16 : stride * es)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(channels), static_cast<cuuint32_t>(rows)};
    const cuuint32_t ones[2] = {1, 1};
    return encode(m, dtype == LA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                  const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- host checks
inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool known_dtype(int32_t d) { return d == LA_DTYPE_BF16 || d == LA_DTYPE_F32; }
inline int dtype_size(int32_t d) { return d == LA_DTYPE_BF16 ? 2 : 4; }
// Whether TMA can move tiles of a [T, D] operand: rows on 16-byte boundaries that do not overlap.
inline bool tileable(const void* p, int64_t stride, int64_t T, int64_t D, int32_t dtype) {
    return T > 0 && aligned_to(p, 16) && (T == 1 || (stride >= D && stride * dtype_size(dtype) % 16 == 0));
}

// A [rows, D] operand: non-null when it has elements, element-aligned, rows that an output does not
// overlap.
inline bool good_rows(const void* p, int64_t stride, int64_t rows, int64_t D, int32_t dtype, bool out) {
    if (rows == 0 || D == 0) return true;
    if (!p || !aligned_to(p, dtype_size(dtype))) return false;
    if (stride < 0) return false;
    return !out || rows == 1 || stride >= D;
}
// Whether `rows` rows of a_row bytes, a_st bytes apart, share memory with rows of b_row bytes.  Operands that lie apart take a
// few comparisons, the same stride two divisions; only rows of one buffer with two strides are gone through.
inline bool bytes_meet(const void* a, int64_t a_st, int64_t a_row, const void* b, int64_t b_st, int64_t b_row, int64_t rows) {
    if (rows == 0) return false;
    int64_t off = static_cast<int64_t>(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a));
    const int64_t last = rows - 1;
    if (off >= last * a_st + a_row || off + last * b_st + b_row <= 0) return false;
    if (rows == 1) return true;
    // whether some i from lo to hi has -b_row < x - i st < a_row
    auto one = [](int64_t x, int64_t st, int64_t a_row, int64_t b_row, int64_t lo, int64_t hi) {
        auto floor_div = [](int64_t n, int64_t d) { return n / d - (n % d < 0); };
        if (st == 0) return -b_row < x && x < a_row;
        return std::max(lo, floor_div(x - a_row, st) + 1) <= std::min(hi, -floor_div(-(x + b_row), st) - 1);
    };
    if (a_st == b_st) return one(off, a_st, a_row, b_row, -last, last);
    if (a_st > b_st) {  // the rows further apart are fewer beside the others
        std::swap(a_st, b_st);
        std::swap(a_row, b_row);
        off = -off;
    }
    // rows of b that lie within a's
    const int64_t first = off < -b_row ? (-b_row - off) / b_st : 0;
    for (int64_t j = first; j <= last; ++j) {
        const int64_t x = off + j * b_st;
        if (x >= last * a_st + a_row) break;
        if (one(x, a_st, a_row, b_row, 0, last)) return true;
    }
    return false;
}
// The same of two operands of D channels.
inline bool rows_meet(const void* a, int64_t a_st, const void* b, int64_t b_st, int64_t rows, int64_t D, int32_t dtype) {
    const int64_t es = dtype_size(dtype);
    return bytes_meet(a, a_st * es, D * es, b, b_st * es, D * es, rows);
}
// Whether a result of rows of D channels shares memory with an optional operand other than by lying exactly over it, element by
// element.  out_size, in_size: bytes of an element.
inline bool clashes(const void* out, int64_t out_st, int64_t out_size, const void* in, int64_t in_st, int64_t in_size, int64_t rows, int64_t D) {
    if (!in || (out == in && out_size == in_size && (out_st == in_st || rows == 1))) return false;
    return bytes_meet(out, out_st * out_size, D * out_size, in, in_st * in_size, D * in_size, rows);
}
// An optional contiguous operand.
inline bool good_optional(const void* p, int32_t dtype) { return !p || aligned_to(p, dtype_size(dtype)); }

inline la_status check_seqs(const void* cu, int32_t bits, int32_t N, int64_t T) {
    if (T < 0 || N < 0) return LA_ERR_INVALID_ARG;
    if (N == 0 && T > 0) return LA_ERR_INVALID_ARG;
    if (T >= (int64_t(1) << 31) - 1024) return LA_ERR_UNSUPPORTED;  // tokens are numbered in 32 bits
    if (bits != 32 && bits != 64) return LA_ERR_INVALID_ARG;
    if (!cu || !aligned_to(cu, bits / 8)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

inline la_status check_gate(int32_t mode, float lb) {
    if (mode == LA_GATE_SOFTPLUS) return LA_ERR_UNSUPPORTED;
    if (mode == LA_GATE_SIGMOID_BOUND) return (lb < 0.f && std::isfinite(lb)) ? LA_OK : LA_ERR_INVALID_ARG;
    return (mode == LA_GATE_LOG || mode == LA_GATE_LOGSIGMOID) ? LA_OK : LA_ERR_INVALID_ARG;
}

inline la_status check_workspace(const void* p, size_t have, size_t need) {
    if (need == 0) return LA_OK;
    return (p && have >= need && aligned_to(p, 256)) ? LA_OK : LA_ERR_WORKSPACE;
}

inline la_status launched() { return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

}  // namespace mixer
}  // namespace la
