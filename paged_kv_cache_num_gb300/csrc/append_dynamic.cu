// append_dynamic.cu -- the append that computes its per-token scales.
//
// Per (token, kv head) row of K and of V: a = max |x_d| over the finite
// elements, s = max(a / qmax, 2^-126), code_d = cast(x_d / s), all in fp32
// with IEEE rounding; the scale goes to the token's slot.
//
// A row is read once: head_dim / 16 lanes hold 16 elements each in
// registers (two 16-byte loads), the maximum is a shuffle reduction among
// them, and each lane stores its 16 codes as one 16-byte piece, which is
// also a piece of the x-vectorised layout.  The same lanes take a token's K
// row and V row of a head: one slot, and twice the bytes in flight.  HBM
// bounds it (60001 int8 tokens of 8 heads: 373 MB in 65 us, 0.84 of the copy
// bandwidth).  With the division instruction it was the issue slots (122 us),
// and still with two refinements per division and a row per lane group (86
// us), so the division is what is kept short:
//
// RN(x / s) through the correctly rounded reciprocal r = RN(1 / s): q = x r,
// then q + (x - q s) r, the residual exact in one FMA (Markstein's
// refinement).  For x and a of at most 11 significant bits and s = RN(a /
// qmax), that is the division's result for every pair of significands and each
// qmax (a test compares all of them; powers of two change nothing).
// The residual must not underflow: s >= 2^-80 keeps it exact for every
// quotient that a cast sees (2^-17 and above).  Rows below that, and rows with
// infinities or NaN, take the division instruction.  The residual's sign is
// such that a zero keeps its own.
#include <type_traits>

#include "append_common.cuh"

namespace pkv {
namespace {

template <int Q8> __device__ __forceinline__ float q8_max()
{
    return Q8 == kE4M3 ? 448.0f : Q8 == kE5M2 ? 57344.0f : 127.0f;
}

__device__ __forceinline__ float quotient(float x, float s, float r)
{
    const float q = x * r;
    return fmaf(-fmaf(q, s, -x), r, q);
}

// 16 elements of a row (words of two) -> 16 codes; returns the row's scale
template <int SRC, int Q8, int LPR>
__device__ __forceinline__ float quantise(const uint32_t (&e)[8], uint32_t (&c)[4])
{
    constexpr uint32_t kInf = SRC == kBF16 ? 0x7f80u : 0x7c00u;
    // magnitudes order like their bits
    uint32_t top2 = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) top2 = __vmaxu2(top2, e[j] & 0x7fff7fffu);
    uint32_t top = max(top2 & 0xffffu, top2 >> 16);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool odd = __any_sync(0xffffffffu, top >= kInf);      // infinities or NaN in one of the warp's rows
    if (odd) {
        top = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t lo = e[j] & 0x7fffu, hi = (e[j] >> 16) & 0x7fffu;
            top = max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const float s = fmaxf(__fdiv_rn(h2f<SRC>(uint16_t(top)), q8_max<Q8>()), 1.17549435e-38f);
    // rows of zeros (and those without a token) divide exactly in any case
    if (!odd && __all_sync(0xffffffffu, s >= 8.271806e-25f || top == 0u)) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float q[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                q[2 * i] = quotient(h2f<SRC>(uint16_t(e[2 * j + i])), s, r);
                q[2 * i + 1] = quotient(h2f<SRC>(uint16_t(e[2 * j + i] >> 16)), s, r);
            }
            if constexpr (Q8 == kI8) {
                // |q| rounds to 127 at most; 1.5 2^23 + q rounds q to an integer, half to even
                uint32_t n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) n[i] = __float_as_uint(__fadd_rn(q[i], 12582912.0f));
                c[j] = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
            } else {
                c[j] = q8x2_encode<Q8>(make_float2(q[0], q[1])) | (q8x2_encode<Q8>(make_float2(q[2], q[3])) << 16);
            }
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            uint32_t ej = e[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) ej = j == i ? e[i] : ej;
            float2 x;
            x.x = __fdiv_rn(h2f<SRC>(uint16_t(ej)), s);
            x.y = __fdiv_rn(h2f<SRC>(uint16_t(ej >> 16)), s);
            const uint32_t two = q8x2_encode<Q8>(x) << (16 * (j & 1));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((j >> 1) == i) c[i] = j & 1 ? c[i] | two : two;
        }
    }
    return s;
}

template <int SRC, bool VEC, int Q8, int LPR>
__global__ void __launch_bounds__(kAppendThreads) append_dynamic_kernel(AppendParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int RPW = 32 / LPR;                   // (token, kv head) pairs per warp
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int64_t warp = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5;
    const int64_t warps = (int64_t(gridDim.x) * blockDim.x) >> 5;
    // A warp's rows: neighbouring heads of a token; in x-vectorised caches, whose
    // 16-byte pieces of neighbouring slots are neighbours, RPW tokens of a head
    // (60001 tokens of 8 heads of 128: 104 -> 77 us).
    const bool tokens = p.c_chunk != 16;
    const int row = lane / LPR;
    Walk2 w(tokens ? warp : warp * RPW + row, tokens ? warps : warps * RPW, p.num_kv_heads);
    for (;; w.next()) {
        const int64_t t = tokens ? w.major * RPW + row : w.major;
        if (!__any_sync(0xffffffffu, t < p.num_tokens)) break;
        const int h = w.minor;
        int64_t blk = 0, off = 0;
        const bool live = t < p.num_tokens && resolve_slot(p, t, blk, off);
        uint32_t e[2][8];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[kv][j] = 0u;
            if (!live) continue;
            const char *src = kv ? p.v_new + t * p.v_src_tok + h * p.v_src_head
                                 : p.k_new + t * p.k_src_tok + h * p.k_src_head;
            if constexpr (VEC) {
                const uint4 *s4 = reinterpret_cast<const uint4 *>(src) + 2 * sub;
                const uint4 a = __ldg(s4), b = __ldg(s4 + 1);
                e[kv][0] = a.x; e[kv][1] = a.y; e[kv][2] = a.z; e[kv][3] = a.w;
                e[kv][4] = b.x; e[kv][5] = b.y; e[kv][6] = b.z; e[kv][7] = b.w;
            } else {
                const uint16_t *s2 = reinterpret_cast<const uint16_t *>(src) + 16 * sub;
#pragma unroll
                for (int j = 0; j < 8; ++j) e[kv][j] = uint32_t(s2[2 * j]) | (uint32_t(s2[2 * j + 1]) << 16);
            }
        }
        const int64_t dst = blk * p.c_blk + off * p.c_slot + h * p.c_head + sub * p.c_chunk;
        const int64_t gs = blk * p.gs_blk + off * p.gs_slot + h * p.gs_head;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint32_t c[4];
            const float s = quantise<SRC, Q8, LPR>(e[kv], c);
            if (live) {
                *reinterpret_cast<uint4 *>((kv ? p.v_cache : p.k_cache) + dst) = make_uint4(c[0], c[1], c[2], c[3]);
                if (sub == 0) (kv ? p.v_gs : p.k_gs)[gs] = s;
            }
        }
    }
}

}  // namespace

cudaError_t launch_append_dynamic(const AppendParams &p, int cache_kind, bool vec16, cudaStream_t s)
{
    if (p.num_tokens == 0 || p.num_kv_heads == 0) return cudaSuccess;
    const int lpr = p.head_dim / 16;
    const int g = grid_for(p.num_tokens * p.num_kv_heads * lpr, kAppendThreads);
    auto kind = [&](auto src_c, auto vec_c, auto lpr_c) -> cudaError_t {
        constexpr int S = decltype(src_c)::value;
        constexpr bool V = decltype(vec_c)::value;
        constexpr int L = decltype(lpr_c)::value;
        if (cache_kind == kE4M3) return launch_pdl(append_dynamic_kernel<S, V, kE4M3, L>, g, kAppendThreads, 0, s, p);
        if (cache_kind == kE5M2) return launch_pdl(append_dynamic_kernel<S, V, kE5M2, L>, g, kAppendThreads, 0, s, p);
        return launch_pdl(append_dynamic_kernel<S, V, kI8, L>, g, kAppendThreads, 0, s, p);
    };
    auto lanes = [&](auto src_c, auto vec_c) -> cudaError_t {
        return lpr == 8 ? kind(src_c, vec_c, std::integral_constant<int, 8>{})
                        : kind(src_c, vec_c, std::integral_constant<int, 4>{});
    };
    auto vec = [&](auto src_c) -> cudaError_t {
        return vec16 ? lanes(src_c, std::true_type{}) : lanes(src_c, std::false_type{});
    };
    return p.src_kind == kBF16 ? vec(std::integral_constant<int, kBF16>{}) : vec(std::integral_constant<int, kF16>{});
}

}  // namespace pkv
