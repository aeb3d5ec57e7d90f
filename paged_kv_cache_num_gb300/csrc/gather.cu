// gather.cu -- cached rows read back through slot_mapping, dequantised.
//
// Row (token, K|V, kv head) is head_dim / 8 pieces of 8 elements: 16 bytes
// of a 16-bit cache, 8 of a one-byte one, 3 of a 3-bit one, and 16 bytes of
// output each.  One warp takes parts of a (token, K|V) row, its lanes over
// the (kv head, piece) pairs, as the appends do.
#include <type_traits>

#include "append_common.cuh"

namespace pkv {
namespace {

// 8 elements of cache kind CK as floats, before the scale; w: the piece's
// bytes (4, 2 or 1 words)
template <int CK>
__device__ __forceinline__ void piece_values(const uint32_t (&w)[4], float (&x)[8])
{
    if constexpr (CK == kF16 || CK == kBF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = h2f<CK>(uint16_t(w[j]));
            x[2 * j + 1] = h2f<CK>(uint16_t(w[j] >> 16));
        }
    } else if constexpr (CK == kI8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = float(int8_t(w[j >> 2] >> (8 * (j & 3))));
    } else if constexpr (CK == kU3) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = float((w[0] >> (3 * j)) & 7u);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 a = fp8x2_to_float2<CK, 0>(w[j]), b = fp8x2_to_float2<CK, 1>(w[j]);
            x[4 * j] = a.x; x[4 * j + 1] = a.y; x[4 * j + 2] = b.x; x[4 * j + 3] = b.y;
        }
    }
}

template <int CK, int OUT, bool VEC, int U>
__global__ void __launch_bounds__(kAppendThreads) gather_kernel(GatherParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const DecodeParams &c = p.c;
    const int lane = threadIdx.x & 31;
    const int groups = c.head_dim / 8;
    const int gsh = (groups & (groups - 1)) == 0 ? __ffs(groups) - 1 : -1;
    const int per = c.num_kv_heads * groups;
    const int parts = (per + 32 * U - 1) / (32 * U);
    const int64_t wstep = (int64_t(gridDim.x) * blockDim.x) >> 5;
    for (Walk2 w((blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5, wstep, parts); w.major < p.num_tokens * 2;
         w.next()) {
        const int64_t t = w.major >> 1;
        const int kv = int(w.major & 1);
        const int64_t slot = p.slot_mapping[t * p.slot_stride];
        if (slot < 0) continue;                                     // warp-uniform
        if (slot >= p.num_slots) {
            if (lane == 0) raise_err(p.err_flag, PKV_DEVERR_SLOT_RANGE);
            continue;
        }
        const int64_t blk = c.block_shift >= 0 ? slot >> c.block_shift : slot / c.block_size;
        const int64_t off = slot - blk * c.block_size;
        const char *src_row = (kv ? c.v_cache : c.k_cache) + blk * c.c_blk + off * c.c_slot;
        char *dst_row = kv ? p.v_out + t * p.v_tok : p.k_out + t * p.k_tok;
        const int64_t dst_head = kv ? p.v_head : p.k_head;
        const int i0 = w.minor * 32 * U + lane;
        uint32_t e[U][4];
        float sc[U], ze[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            if (i >= per) continue;
            const int h = gsh >= 0 ? i >> gsh : i / groups, g = i - h * groups;
            const char *src = src_row + h * c.c_head;
            sc[u] = 1.0f;
            ze[u] = 0.0f;
            if constexpr (CK == kF16 || CK == kBF16) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + g * c.c_chunk));
                e[u][0] = v.x; e[u][1] = v.y; e[u][2] = v.z; e[u][3] = v.w;
            } else if constexpr (CK == kU3) {
                const uint8_t *b = reinterpret_cast<const uint8_t *>(src) + 3 * g;
                e[u][0] = uint32_t(__ldg(b)) | (uint32_t(__ldg(b + 1)) << 8) | (uint32_t(__ldg(b + 2)) << 16);
                sc[u] = __half2float(__ushort_as_half(__ldg((kv ? c.v_qs : c.k_qs) + blk * c.m_blk + off * c.m_slot + h * c.m_head)));
                ze[u] = float(__ldg((kv ? c.v_qz : c.k_qz) + blk * c.z_blk + off * c.z_slot + h * c.z_head));
            } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + (g >> 1) * c.c_chunk + 8 * (g & 1)));
                e[u][0] = v.x; e[u][1] = v.y;
                sc[u] = c.scale_mode == 0 ? __ldg((kv ? c.v_scale : c.k_scale) + h)
                                          : __ldg((kv ? c.v_gs : c.k_gs) + blk * c.gs_blk + off * c.gs_slot + h * c.gs_head);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            if (i >= per) continue;
            const int h = gsh >= 0 ? i >> gsh : i / groups, g = i - h * groups;
            uint32_t o[4];
            if constexpr (CK == OUT) {              // same 16-bit type: the bits
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = e[u][j];
            } else {
                float x[8];
                piece_values<CK>(e[u], x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = uint32_t(f2h<OUT>((x[2 * j] - ze[u]) * sc[u])) |
                           (uint32_t(f2h<OUT>((x[2 * j + 1] - ze[u]) * sc[u])) << 16);
            }
            uint16_t *dst = reinterpret_cast<uint16_t *>(dst_row + h * dst_head) + 8 * g;
            if constexpr (VEC) {
                *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) dst[j] = uint16_t(o[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

}  // namespace

cudaError_t launch_gather(const GatherParams &p, int cache_kind, int out_kind, cudaStream_t s)
{
    if (p.num_tokens == 0 || p.c.num_kv_heads == 0) return cudaSuccess;
    const int per = p.c.num_kv_heads * (p.c.head_dim / 8);
    const int64_t rows = p.num_tokens * 2;
    const bool one = rows * ((per + 127) / 128) < int64_t(sm_count_current_device()) * 8;
    const int U = one ? 1 : 4;
    const int g = grid_for(rows * ((per + 32 * U - 1) / (32 * U)) * 32, kAppendThreads);
    auto go = [&](auto ck_c, auto out_c, auto vec_c) -> cudaError_t {
        constexpr int CK = decltype(ck_c)::value;
        constexpr int OUT = decltype(out_c)::value;
        constexpr bool V = decltype(vec_c)::value;
        return one ? launch_pdl(gather_kernel<CK, OUT, V, 1>, g, kAppendThreads, 0, s, p)
                   : launch_pdl(gather_kernel<CK, OUT, V, 4>, g, kAppendThreads, 0, s, p);
    };
    auto out = [&](auto ck_c) -> cudaError_t {
        using HF = std::integral_constant<int, kF16>;
        using BF = std::integral_constant<int, kBF16>;
        if (out_kind == kBF16) return p.vec16 ? go(ck_c, BF{}, std::true_type{}) : go(ck_c, BF{}, std::false_type{});
        return p.vec16 ? go(ck_c, HF{}, std::true_type{}) : go(ck_c, HF{}, std::false_type{});
    };
    switch (cache_kind) {
    case kF16: return out(std::integral_constant<int, kF16>{});
    case kBF16: return out(std::integral_constant<int, kBF16>{});
    case kE4M3: return out(std::integral_constant<int, kE4M3>{});
    case kE5M2: return out(std::integral_constant<int, kE5M2>{});
    case kI8: return out(std::integral_constant<int, kI8>{});
    default: return out(std::integral_constant<int, kU3>{});
    }
}

}  // namespace pkv
