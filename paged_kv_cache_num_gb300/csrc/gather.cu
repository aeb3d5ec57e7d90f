// gather.cu -- cached rows read back through slot_mapping, dequantised.
//
// A row (token, K|V, kv head) is read in pieces of EPP elements: 16 bytes of
// a 16-bit cache (8) or a one-byte one (16; 8 where head_dim is no multiple
// of 16), 16 or 12 bytes of a 4- or 3-bit one (32).  One warp takes parts of a
// (token, K|V) row, its lanes over the (kv head, piece) pairs, as the appends
// do, all of a lane's loads before its stores.  Bound by HBM.  A 3-bit row has
// only eight values: a lane forms them once, (u - z) s rounded, and looks its
// codes up by byte permutes of their low and high bytes.
#include <type_traits>

#include "append_common.cuh"
#include "tc_ptx.cuh"

namespace pkv {
namespace {

// two elements -> two of the output type, times the scale
template <int CK, int OUT>
__device__ __forceinline__ uint32_t pair_out(uint32_t w, float s)
{
    float x, y;
    if constexpr (CK == kF16 || CK == kBF16) {      // w: two 16-bit elements
        x = h2f<CK>(uint16_t(w));
        y = h2f<CK>(uint16_t(w >> 16));
    } else if constexpr (CK == kI8) {               // the low two bytes
        x = float(int8_t(w)) * s;
        y = float(int8_t(w >> 8)) * s;
    } else {
        const float2 v = fp8x2_to_float2<CK, 0>(w);
        x = v.x * s;
        y = v.y * s;
    }
    return uint32_t(f2h<OUT>(x)) | (uint32_t(f2h<OUT>(y)) << 16);
}

// elements of a piece -> N words of the output
template <int CK, int OUT, int N>
__device__ __forceinline__ void piece_out(const uint32_t (&w)[4], float s, float z, uint32_t (&o)[N])
{
    if constexpr (CK == OUT) {                      // same 16-bit type: the bits
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = w[j];
    } else if constexpr (CK == kF16 || CK == kBF16) {
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = pair_out<CK, OUT>(w[j], 1.0f);
    } else if constexpr (CK == kU4) {
        // u - z exactly as f16; times s: of an f16 output one rounding by itself (the
        // product of 5 and 11 bits is exact in fp32 too, so both round alike)
        const uint32_t zz = __half_as_ushort(__float2half_rn(-1024.0f - z)) * 0x10001u;
        const __half2 ss = __float2half2_rn(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t p[4];
            u4x8_to_f16(w[j], zz, p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 x = *reinterpret_cast<const __half2 *>(&p[i]);
                if constexpr (OUT == kF16) {
                    const __half2 y = __hmul2(x, ss);
                    o[4 * j + i] = *reinterpret_cast<const uint32_t *>(&y);
                } else {
                    const float2 y = __half22float2(x);
                    const __nv_bfloat162 r = __floats2bfloat162_rn(y.x * s, y.y * s);
                    o[4 * j + i] = *reinterpret_cast<const uint32_t *>(&r);
                }
            }
        }
    } else if constexpr (CK == kU3) {
        uint32_t v[4], lo[2], hi[2];                // the row's eight values, two per word
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = uint32_t(f2h<OUT>((float(2 * u) - z) * s)) | (uint32_t(f2h<OUT>((float(2 * u + 1) - z) * s)) << 16);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            lo[u] = __byte_perm(v[2 * u], v[2 * u + 1], 0x6420);
            hi[u] = __byte_perm(v[2 * u], v[2 * u + 1], 0x7531);
        }
        const uint32_t f[4] = {w[0], __funnelshift_r(w[0], w[1], 24), __funnelshift_r(w[1], w[2], 16), w[2] >> 8};
#pragma unroll
        for (int j = 0; j < 8; ++j) {               // four codes, one per hex digit of the selector
            const uint32_t x = f[j >> 1] >> (12 * (j & 1));
            const uint32_t sel = (x & 7u) | ((x << 1) & 0x70u) | ((x << 2) & 0x700u) | ((x << 3) & 0x7000u);
            const uint32_t a = __byte_perm(lo[0], lo[1], sel), b = __byte_perm(hi[0], hi[1], sel);
            o[2 * j] = __byte_perm(a, b, 0x5140);
            o[2 * j + 1] = __byte_perm(a, b, 0x7362);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = pair_out<CK, OUT>(w[j >> 1] >> (16 * (j & 1)), s);
    }
}

template <int CK, int OUT, int EPP, int U>
__global__ void __launch_bounds__(kAppendThreads) gather_kernel(GatherParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const DecodeParams &c = p.c;
    const int lane = threadIdx.x & 31;
    const int groups = c.head_dim / EPP;
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
            if constexpr (is_packed(CK)) {
                sc[u] = __half2float(__ushort_as_half(__ldg((kv ? c.v_qs : c.k_qs) + blk * c.m_blk + off * c.m_slot + h * c.m_head)));
                ze[u] = float(__ldg((kv ? c.v_qz : c.k_qz) + blk * c.z_blk + off * c.z_slot + h * c.z_head));
            }
            if constexpr (CK == kU3) {
                src += 12 * g;
                if (p.word_rows) {
#pragma unroll
                    for (int j = 0; j < 3; ++j) e[u][j] = __ldg(reinterpret_cast<const uint32_t *>(src) + j);
                } else {                            // rows off the 4-byte boundary
#pragma unroll
                    for (int j = 0; j < 12; ++j)
                        e[u][j >> 2] = (j & 3 ? e[u][j >> 2] : 0u) |
                                       uint32_t(__ldg(reinterpret_cast<const uint8_t *>(src) + j)) << (8 * (j & 3));
                }
            } else if constexpr (EPP == 8 && is_q8(CK)) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + (g >> 1) * c.c_chunk + 8 * (g & 1)));
                e[u][0] = v.x; e[u][1] = v.y;
            } else {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + g * c.c_chunk));
                e[u][0] = v.x; e[u][1] = v.y; e[u][2] = v.z; e[u][3] = v.w;
            }
            if constexpr (is_q8(CK))
                sc[u] = c.scale_mode == 0 ? __ldg((kv ? c.v_scale : c.k_scale) + h)
                                          : __ldg((kv ? c.v_gs : c.k_gs) + blk * c.gs_blk + off * c.gs_slot + h * c.gs_head);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            if (i >= per) continue;
            const int h = gsh >= 0 ? i >> gsh : i / groups, g = i - h * groups;
            uint32_t o[EPP / 2];
            piece_out<CK, OUT>(e[u], sc[u], ze[u], o);
            uint16_t *dst = reinterpret_cast<uint16_t *>(dst_row + h * dst_head) + EPP * g;
            if (EPP >= 16 && p.align == 32) {
#pragma unroll
                for (int j = 0; j + 8 <= EPP / 2; j += 8) tc::st_global32(dst + 2 * j, o + j);
            } else if (p.align >= 16) {
#pragma unroll
                for (int j = 0; j < EPP / 2; j += 4)
                    *reinterpret_cast<uint4 *>(dst + 2 * j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < EPP; ++j) dst[j] = uint16_t(o[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

}  // namespace

cudaError_t launch_gather(const GatherParams &p, int cache_kind, int out_kind, cudaStream_t s)
{
    if (p.num_tokens == 0 || p.c.num_kv_heads == 0) return cudaSuccess;
    const int64_t rows = p.num_tokens * 2;
    auto go = [&](auto ck_c, auto out_c, auto epp_c) -> cudaError_t {
        constexpr int CK = decltype(ck_c)::value;
        constexpr int OUT = decltype(out_c)::value;
        constexpr int EPP = decltype(epp_c)::value;
        const int per = p.c.num_kv_heads * (p.c.head_dim / EPP);
        // pieces per lane: four where a (token, K|V) row has them and that leaves every
        // SM several warps, else two, else one
        auto warps = [&](int U) { return rows * ((per + 32 * U - 1) / (32 * U)); };
        const int64_t enough = int64_t(sm_count_current_device()) * 8;
        const int U = per > 64 && warps(4) >= enough ? 4 : per > 32 && warps(2) >= enough ? 2 : 1;
        const int g = grid_for(warps(U) * 32, kAppendThreads);
        return U == 4   ? launch_pdl(gather_kernel<CK, OUT, EPP, 4>, g, kAppendThreads, 0, s, p)
               : U == 2 ? launch_pdl(gather_kernel<CK, OUT, EPP, 2>, g, kAppendThreads, 0, s, p)
                        : launch_pdl(gather_kernel<CK, OUT, EPP, 1>, g, kAppendThreads, 0, s, p);
    };
    auto out = [&](auto ck_c, auto epp_c) -> cudaError_t {
        return out_kind == kBF16 ? go(ck_c, std::integral_constant<int, kBF16>{}, epp_c)
                                 : go(ck_c, std::integral_constant<int, kF16>{}, epp_c);
    };
    using E8 = std::integral_constant<int, 8>;
    using E16 = std::integral_constant<int, 16>;
    auto q8 = [&](auto ck_c) -> cudaError_t { return p.c.head_dim % 16 == 0 ? out(ck_c, E16{}) : out(ck_c, E8{}); };
    switch (cache_kind) {
    case kF16: return out(std::integral_constant<int, kF16>{}, E8{});
    case kBF16: return out(std::integral_constant<int, kBF16>{}, E8{});
    case kE4M3: return q8(std::integral_constant<int, kE4M3>{});
    case kE5M2: return q8(std::integral_constant<int, kE5M2>{});
    case kI8: return q8(std::integral_constant<int, kI8>{});
    case kU4: return out(std::integral_constant<int, kU4>{}, std::integral_constant<int, 32>{});
    default: return out(std::integral_constant<int, kU3>{}, std::integral_constant<int, 32>{});
    }
}

}  // namespace pkv
