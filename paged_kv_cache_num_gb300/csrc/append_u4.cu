// append_u4.cu -- append into 4-bit caches: per (token, kv head) row of K and
// of V, in fp32 with IEEE rounding,
//   lo = min(0, min x), hi = max(0, max x), s = fp16((hi - lo) / 15),
//   z = clamp(rint(-lo / s), 0, 15), code_d = clamp(rint(x_d / s) + z, 0, 15).
// The range takes zero in, so z is never cut off and a row of equal numbers
// keeps its value.
//
// A lane takes 16 elements (32 source bytes -> two words of codes), so a row is 8
// lanes at head_dim 128 and 4 at 64; one warp takes parts of a (token, K|V) row,
// its lanes over the (kv head, 16 elements) pieces, as the one-byte appends do.
// The extremes of a row go through its lanes as one word, (min, -max) in 16 bits
// each: exact, the elements being 16-bit numbers.  40001 f16 tokens of 8 heads of 128
// (207 MB) take 55 us, 0.55 of the copy bandwidth: 300 instructions for a lane's 16
// elements, of which an SM sub-partition issues 0.77 a cycle (8 elements a lane and the
// rounding instruction instead of an addition: 79 us).
#include <type_traits>

#include "append_common.cuh"

namespace pkv {
namespace {

// Whole rows per warp and step: the lanes of a row stay together (head_dim /
// 16 divides 32 and a part begins at a multiple of 32 pieces).
template <int SRC, bool VEC, int D, int U>
__global__ void __launch_bounds__(kAppendThreads) append_u4_kernel(AppendParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int LPR = D / 16;                     // lanes of a row
    const int lane = threadIdx.x & 31;
    const int per = p.num_kv_heads * LPR;           // pieces per (token, K|V)
    const int parts = (per + 32 * U - 1) / (32 * U);
    const int64_t wstep = (int64_t(gridDim.x) * blockDim.x) >> 5;
    for (Walk2 w((blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5, wstep, parts); w.major < p.num_tokens * 2;
         w.next()) {
        const int64_t t = w.major >> 1;
        const int kv = int(w.major & 1);
        int64_t blk, off;
        if (!resolve_slot(p, t, blk, off, kv == 0 && w.minor == 0 && lane == 0)) continue;     // warp-uniform
        const char *src_row = kv ? p.v_new + t * p.v_src_tok : p.k_new + t * p.k_src_tok;
        const int64_t src_head = kv ? p.v_src_head : p.k_src_head;
        char *dst_row = (kv ? p.v_cache : p.k_cache) + blk * p.c_blk + off * p.c_slot;
        uint16_t *qs = (kv ? p.v_qs : p.k_qs) + blk * p.m_blk + off * p.m_slot;
        uint8_t *qz = (kv ? p.v_qz : p.k_qz) + blk * p.z_blk + off * p.z_slot;
        const int i0 = w.minor * 32 * U + lane;
        uint32_t e[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u, h = i / LPR, c = i % LPR;
#pragma unroll
            for (int j = 0; j < 8; ++j) e[u][j] = 0u;
            if (i >= per) continue;
            const uint16_t *src = reinterpret_cast<const uint16_t *>(src_row + h * src_head) + 16 * c;
            if constexpr (VEC) {
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src)), b = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
                e[u][0] = a.x; e[u][1] = a.y; e[u][2] = a.z; e[u][3] = a.w;
                e[u][4] = b.x; e[u][5] = b.y; e[u][6] = b.z; e[u][7] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) e[u][j] = uint32_t(src[2 * j]) | (uint32_t(src[2 * j + 1]) << 16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u, h = i / LPR, c = i % LPR;
            const RowU4<2> r = row_u4<SRC, LPR, 2>(e[u]);
            if (i >= per) continue;
            *(reinterpret_cast<uint2 *>(dst_row + h * p.c_head) + c) = make_uint2(r.codes[0], r.codes[1]);
            if (c == 0) {
                qs[h * p.m_head] = r.scale;
                qz[h * p.z_head] = uint8_t(r.zero);
            }
        }
    }
}

}  // namespace

cudaError_t launch_append_u4(const AppendParams &p, bool vec16, cudaStream_t s)
{
    const int per = p.num_kv_heads * (p.head_dim / 16);
    if (p.num_tokens == 0 || per == 0) return cudaSuccess;
    // two pieces per lane where a (token, K|V) row has them and every SM still gets
    // several warps, else one (more, shorter warps)
    auto warps = [&](int U) { return p.num_tokens * 2 * ((per + 32 * U - 1) / (32 * U)); };
    const bool one = per <= 32 || warps(2) < int64_t(sm_count_current_device()) * 8;
    const int g = grid_for(warps(one ? 1 : 2) * 32, kAppendThreads);
    auto go = [&](auto src_c, auto vec_c) -> cudaError_t {
        constexpr int S = decltype(src_c)::value;
        constexpr bool V = decltype(vec_c)::value;
        if (p.head_dim == 128)
            return one ? launch_pdl(append_u4_kernel<S, V, 128, 1>, g, kAppendThreads, 0, s, p)
                       : launch_pdl(append_u4_kernel<S, V, 128, 2>, g, kAppendThreads, 0, s, p);
        return one ? launch_pdl(append_u4_kernel<S, V, 64, 1>, g, kAppendThreads, 0, s, p)
                   : launch_pdl(append_u4_kernel<S, V, 64, 2>, g, kAppendThreads, 0, s, p);
    };
    using BF = std::integral_constant<int, kBF16>;
    using HF = std::integral_constant<int, kF16>;
    if (p.src_kind == kBF16) return vec16 ? go(BF{}, std::true_type{}) : go(BF{}, std::false_type{});
    return vec16 ? go(HF{}, std::true_type{}) : go(HF{}, std::false_type{});
}

}  // namespace pkv
