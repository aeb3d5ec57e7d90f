// norm_rope.cu -- the norm of each query and key head and its rotation by
// position, in one pass over the projection's output; the rotated keys and the
// values go into the cache in the same pass, stored as the appends store them.
//
// Per head row x of head_dim elements, in fp32, rounded once:
//   y_d = x_d / sqrt(mean x^2 + eps) w_d           (without weights y = x)
//   (y_i, y_j) -> (y_i cos - y_j sin, y_j cos + y_i sin),  i < rot / 2,
// with j = i + rot / 2, or (interleaved) the pair 2i, 2i + 1; elements from rot
// on stay.  cos and sin are the row of a table that the token's position names.
//
// One warp takes a token, or a part of its query, key or value rows, 8 elements (16
// bytes) a lane, U row groups at a time, their loads before the arithmetic: the
// products of the weights and the table's row are made once for all of them.  A row is 16 or 8
// neighbouring lanes: its sum of squares is log2 of that in shuffles, the other
// half of a rotated pair four more (of the 16-bit source; the norm's factor is the
// row's, and the other's weight is in the table's products).
// 20011 tokens, 32 q and 8 kv heads of 128, bf16 (497 MB): 98 us, 0.75 of the copy
// bandwidth (the products made for every four row groups 117, at 101 registers 149);
// what is left is latency: 24 warps an SM with 2 KB each on the way.  A decode step's 64
// tokens take 3.4 us on the device.
#include <type_traits>

#include "append_common.cuh"

namespace pkv {
namespace {

// 3-bit row of LPR lanes with 8 elements each: this lane's 24 bits of codes
template <int SRC, int LPR>
__device__ __forceinline__ RowU4<1> row_u3(const uint32_t (&e)[4])
{
    uint32_t mn = min2_16<SRC>(min2_16<SRC>(e[0], e[1]), min2_16<SRC>(e[2], e[3]));
    uint32_t mx = max2_16<SRC>(max2_16<SRC>(e[0], e[1]), max2_16<SRC>(e[2], e[3]));
    float lo = fminf(h2f<SRC>(uint16_t(mn)), h2f<SRC>(uint16_t(mn >> 16)));
    float hi = fmaxf(h2f<SRC>(uint16_t(mx)), h2f<SRC>(uint16_t(mx >> 16)));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    uint16_t sbits = __half_as_ushort(__float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 7.0f)));
    if ((sbits & 0x7fff) == 0x7c00) sbits = 0x7bff;
    const float s = __half2float(__ushort_as_half(sbits));
    const float rs = s != 0.0f ? __frcp_rn(s) : 0.0f;
    const float z = s != 0.0f ? fminf(fmaxf(rintf(row_quotient(-lo, s, rs)), 0.0f), 7.0f) : 0.0f;
    float f = 0.0f;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float x = h2f<SRC>(uint16_t(i & 1 ? e[i >> 1] >> 16 : e[i >> 1]));
        f = fmaf(f, 8.0f, fminf(fmaxf(__fadd_rn(rintf(row_quotient(x, s, rs)), z), 0.0f), 7.0f));
    }
    return {{uint32_t(f)}, sbits, uint32_t(z)};
}

// the scale that kv_append_dynamic computes for a row of LPR lanes
template <int SRC, int Q8, int LPR>
__device__ __forceinline__ float dynamic_scale(const uint32_t (&e)[4])
{
    constexpr uint32_t kInf = SRC == kBF16 ? 0x7f80u : 0x7c00u;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = e[j] & 0x7fffu, hi = (e[j] >> 16) & 0x7fffu;
        top = max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));      // the largest finite element
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    constexpr float qmax = Q8 == kE4M3 ? 448.0f : Q8 == kE5M2 ? 57344.0f : 127.0f;
    return fmaxf(__fdiv_rn(h2f<SRC>(uint16_t(top)), qmax), 1.17549435e-38f);
}

// where a lane's 8 elements lie in a cached row (piece c of head_dim / 8)
template <int CK>
__device__ __forceinline__ int64_t piece_offset(const AppendParams &p, int c)
{
    if constexpr (CK == kF16 || CK == kBF16) return c * p.c_chunk;
    else if constexpr (is_q8(CK)) return (c >> 1) * p.c_chunk + 8 * (c & 1);
    else return CK == kU4 ? 4 * c : 3 * c;
}

// 8 elements (pairs in order) of piece c of head h's row, to their place `to` in the cache, the
// token's being (blk, off).  Every lane calls it; `on` lanes store.
template <int SRC, int CK, int LPR>
__device__ __forceinline__ void store_piece(const AppendParams &p, char *to, bool v, int64_t blk, int64_t off, int h, int c, bool on, const uint32_t (&e)[4])
{
    if constexpr (CK == kF16 || CK == kBF16) {
        if (on) *reinterpret_cast<uint4 *>(to) = make_uint4(e[0], e[1], e[2], e[3]);
    } else if constexpr (is_q8(CK)) {
        float scale = 1.0f;
        if (p.scale_mode == 2) {
            scale = dynamic_scale<SRC, CK, LPR>(e);
            if (on && c == 0) (v ? p.v_gs : p.k_gs)[blk * p.gs_blk + off * p.gs_slot + h * p.gs_head] = scale;
        } else if (on) {
            scale = p.scale_mode == 0 ? (v ? p.v_scale : p.k_scale)[h] : (v ? p.v_gs : p.k_gs)[blk * p.gs_blk + h * p.gs_head];
        }
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 x;
            x.x = __fdiv_rn(h2f<SRC>(uint16_t(e[j])), scale);
            x.y = __fdiv_rn(h2f<SRC>(uint16_t(e[j] >> 16)), scale);
            const uint32_t two = q8x2_encode<CK>(x);
            w[j >> 1] = j & 1 ? w[j >> 1] | (two << 16) : two;
        }
        if (on) *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    } else {
        RowU4<1> r;
        if constexpr (CK == kU4) r = row_u4<SRC, LPR, 1>(e);
        else r = row_u3<SRC, LPR>(e);
        if (!on) return;
        if constexpr (CK == kU4) {
            *reinterpret_cast<uint32_t *>(to) = r.codes[0];
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j) to[j] = char(r.codes[0] >> (8 * j));
        }
        if (c == 0) {
            (v ? p.v_qs : p.k_qs)[blk * p.m_blk + off * p.m_slot + h * p.m_head] = r.scale;
            (v ? p.v_qz : p.k_qz)[blk * p.z_blk + off * p.z_slot + h * p.z_head] = uint8_t(r.zero);
        }
    }
}

// 8 weights from element d on
__device__ __forceinline__ void load_weights(const NormRopeParams &p, const void *w, int d, float (&o)[8])
{
    if (p.weight_kind == PKV_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __ldg(static_cast<const float *>(w) + d + i);
    } else if (p.weight_vec) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + d));
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t v = uint16_t(x[i >> 1] >> (16 * (i & 1)));
            o[i] = p.weight_kind == kBF16 ? h2f<kBF16>(v) : h2f<kF16>(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t u = __ldg(static_cast<const uint16_t *>(w) + d + i);
            o[i] = p.weight_kind == kBF16 ? h2f<kBF16>(u) : h2f<kF16>(u);
        }
    }
}

// CK: the cache's kind; 0: keys to k_out, and no values
template <int SRC, int CK, int D, int U>
__global__ void __launch_bounds__(kAppendThreads, 3) norm_rope_kernel(NormRopeParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int LPR = D / 8;                      // lanes of a row
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int hk = p.a.num_kv_heads;
    // parts of a token: of its query rows, its key rows, its value rows
    const int per_part = 32 * U / LPR;              // rows
    const int parts_q = (p.num_heads + per_part - 1) / per_part, parts_k = (hk + per_part - 1) / per_part;
    const int half = p.rot / 2;
    const bool turned = 8 * sub < p.rot;
    // the lane that holds the other elements of this lane's pairs, where they are half a rotation apart
    const int other = p.interleaved || !turned ? lane : 8 * sub < half ? lane + half / 8 : lane - half / 8;
    const float sign = 8 * sub < half ? -1.0f : 1.0f;
    const int64_t wstep = (int64_t(gridDim.x) * blockDim.x) >> 5;
    // an item is a token, or, of few tokens, a part of one
    const int parts = parts_q + (CK ? 2 : 1) * parts_k;
    Walk2 w((blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5, wstep, p.whole ? 1 : parts);
    // the position and slot of an item are loaded while the one before is worked on
    int32_t pos_next = -1;
    int64_t slot_next = -1;
    auto fetch = [&]() {
        if (w.major >= p.a.num_tokens) return;
        pos_next = p.pos[w.major * p.pos_stride];
        if (CK && (p.whole || w.minor >= parts_q)) slot_next = p.a.slot_mapping[w.major * p.a.slot_stride];
    };
    fetch();
    while (w.major < p.a.num_tokens) {
        const int64_t t = w.major, slot = slot_next;
        const int minor = w.minor;
        const int32_t pos = pos_next;
        w.next();
        fetch();
        if (pos < 0) continue;                      // a padding token
        if (pos >= p.max_pos) {
            if (lane == 0) raise_err(p.a.err_flag, PKV_DEVERR_POS_RANGE);
            continue;
        }
        int part = p.whole ? 0 : minor, end = p.whole ? parts : minor + 1;
        int64_t blk = 0, off = 0;
        if (CK && end > parts_q && !place_slot(p.a, slot, blk, off)) end = min(end, parts_q);      // queries alone
        // a row's element becomes r (x a + y b): x itself, y the other of its pair, a and b
        // weights times cosine and signed sine, r what the norm divides by
        float a[8], b[8];
        for (bool first = true; part < end; ++part, first = false) {
            const int what = part < parts_q ? 0 : part < parts_q + parts_k ? 1 : 2;             // queries, keys, values
            const int heads = what == 0 ? p.num_heads : hk;
            const int h0 = (part - (what == 0 ? 0 : what == 1 ? parts_q : parts_q + parts_k)) * per_part + lane / LPR;
            // this lane's place in the first row group, and how far the next one's is
            const int64_t src_head = what == 0 ? p.q_head : what == 1 ? p.a.k_src_head : p.a.v_src_head;
            const char *src = (what == 0 ? p.q + t * p.q_tok : what == 1 ? p.a.k_new + t * p.a.k_src_tok : p.a.v_new + t * p.a.v_src_tok) +
                              h0 * src_head + 16 * sub;
            const int64_t src_step = 32 / LPR * src_head;
            uint32_t e[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * (32 / LPR);
                e[u][0] = e[u][1] = e[u][2] = e[u][3] = 0u;
                const uint16_t *s = reinterpret_cast<const uint16_t *>(src);
                src += src_step;
                if (h >= heads) continue;
                if (p.vec) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(s);        // (the output may be the same memory)
                    e[u][0] = x.x; e[u][1] = x.y; e[u][2] = x.z; e[u][3] = x.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[u][j] = uint32_t(s[2 * j]) | (uint32_t(s[2 * j + 1]) << 16);
                }
            }
            if (what < 2) {
                const void *weight = what == 0 ? p.q_weight : p.k_weight;
                const bool norm = weight != nullptr;
                if (first || part == parts_q) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] = 1.0f;
                        b[i] = 0.0f;
                    }
                    if (turned) {                           // pairs 4 sub .. + 3 of 8 sub .. + 7, or those of 8 sub modulo rot / 2
                        const float *row = p.cos_sin + int64_t(pos) * p.cs_row + (p.interleaved ? 4 * sub : 8 * sub < half ? 8 * sub : 8 * sub - half);
                        const float4 c0 = __ldg(reinterpret_cast<const float4 *>(row)), s0 = __ldg(reinterpret_cast<const float4 *>(row + half));
                        if (p.interleaved) {
                            const float c4[4] = {c0.x, c0.y, c0.z, c0.w}, s4[4] = {s0.x, s0.y, s0.z, s0.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                a[i] = c4[i >> 1];
                                b[i] = i & 1 ? s4[i >> 1] : -s4[i >> 1];
                            }
                        } else {
                            const float4 c1 = __ldg(reinterpret_cast<const float4 *>(row) + 1), s1 = __ldg(reinterpret_cast<const float4 *>(row + half) + 1);
                            const float c8[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}, s8[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                a[i] = c8[i];
                                b[i] = sign * s8[i];
                            }
                        }
                    }
                    if (norm) {
                        float w[8];
                        load_weights(p, weight, 8 * sub, w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) a[i] *= w[i];
                        if (!p.interleaved) load_weights(p, weight, 8 * (sub + other - lane), w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) b[i] *= p.interleaved ? w[i ^ 1] : w[i];
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[8], y[8], r = 1.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 v = h2f2<SRC>(e[u][j]);
                        x[2 * j] = v.x;
                        x[2 * j + 1] = v.y;
                    }
                    if (norm) {
                        float ss = 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                        r = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
                    }
                    if (p.interleaved) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 v = h2f2<SRC>(__shfl_sync(0xffffffffu, e[u][j], other));
                            y[2 * j] = v.x;
                            y[2 * j + 1] = v.y;
                        }
                    }
                    if (turned) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], a[i], y[i] * b[i]);
                    } else if (norm) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] *= a[i];
                    }
                    if (norm || turned)                 // (else the source's bits)
#pragma unroll
                        for (int j = 0; j < 4; ++j) e[u][j] = f2h2<SRC>(r * x[2 * j], r * x[2 * j + 1]);
                }
            }
            if (CK && what > 0) {
                char *to = (what == 2 ? p.a.v_cache : p.a.k_cache) + blk * p.a.c_blk + off * p.a.c_slot + h0 * p.a.c_head + piece_offset<CK>(p.a, sub);
#pragma unroll
                for (int u = 0; u < U; ++u, to += 32 / LPR * p.a.c_head) {
                    const int h = h0 + u * (32 / LPR);
                    store_piece<SRC, CK, LPR>(p.a, to, what == 2, blk, off, h, sub, h < heads, e[u]);
                }
            } else {
                const int64_t head = what == 0 ? p.qo_head : p.ko_head;
                char *to = (what == 0 ? p.q_out + t * p.qo_tok : p.k_out + t * p.ko_tok) + h0 * head + 16 * sub;
#pragma unroll
                for (int u = 0; u < U; ++u, to += 32 / LPR * head) {
                    if (h0 + u * (32 / LPR) >= heads) continue;
                    uint16_t *o = reinterpret_cast<uint16_t *>(to);
                    if (p.out_vec) {
                        *reinterpret_cast<uint4 *>(o) = make_uint4(e[u][0], e[u][1], e[u][2], e[u][3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = uint16_t(e[u][j >> 1] >> (16 * (j & 1)));
                    }
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int cache_kind, cudaStream_t s)
{
    if (p.a.num_tokens == 0) return cudaSuccess;
    const int lpr = p.a.head_dim / 8;
    auto parts = [&](int U) {
        const int rows = 32 * U / lpr;
        return (p.num_heads + rows - 1) / rows + (cache_kind ? 2 : 1) * ((p.a.num_kv_heads + rows - 1) / rows);
    };
    // four row groups at a time where that still gives every SM several warps, else one; and
    // whole tokens, one after another, where every SM gets its fill of them
    const int64_t sms = sm_count_current_device();
    const bool one = p.a.num_tokens * parts(4) < sms * 8;
    int n = parts(one ? 1 : 4);
    if (n == 0) return cudaSuccess;
    p.whole = p.a.num_tokens >= sms * 32;
    if (p.whole) n = 1;
    const int g = grid_for(p.a.num_tokens * n * 32, kAppendThreads);
    auto go = [&](auto src_c, auto ck_c, auto d_c) -> cudaError_t {
        constexpr int S = decltype(src_c)::value, CK = decltype(ck_c)::value, D = decltype(d_c)::value;
        return one ? launch_pdl(norm_rope_kernel<S, CK, D, 1>, g, kAppendThreads, 0, s, p)
                   : launch_pdl(norm_rope_kernel<S, CK, D, 4>, g, kAppendThreads, 0, s, p);
    };
    auto by_dim = [&](auto src_c, auto ck_c) -> cudaError_t {
        return p.a.head_dim == 128 ? go(src_c, ck_c, std::integral_constant<int, 128>{}) : go(src_c, ck_c, std::integral_constant<int, 64>{});
    };
    auto by_kind = [&](auto src_c) -> cudaError_t {
        switch (cache_kind) {
        case 0: return by_dim(src_c, std::integral_constant<int, 0>{});
        case kF16:
        case kBF16: return by_dim(src_c, src_c);
        case kE4M3: return by_dim(src_c, std::integral_constant<int, kE4M3>{});
        case kE5M2: return by_dim(src_c, std::integral_constant<int, kE5M2>{});
        case kI8: return by_dim(src_c, std::integral_constant<int, kI8>{});
        case kU4: return by_dim(src_c, std::integral_constant<int, kU4>{});
        default: return by_dim(src_c, std::integral_constant<int, kU3>{});
        }
    };
    return p.a.src_kind == kBF16 ? by_kind(std::integral_constant<int, kBF16>{}) : by_kind(std::integral_constant<int, kF16>{});
}

}  // namespace pkv
