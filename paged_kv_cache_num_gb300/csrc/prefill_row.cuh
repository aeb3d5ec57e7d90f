// prefill_row.cuh -- one output row of the prefill attention by one warp,
// straight from the definition: each lane owns head_dim / 32 elements, the
// keys are taken one at a time, fp32 throughout.
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace {

// This lane's EPL elements (e0 .. e0 + EPL - 1) of one cached row, dequantised.
template <int CK, int EPL>
__device__ __forceinline__ void cached_elems(const DecodeParams &p, bool v, int64_t blk, int off, int h, int e0,
                                             float (&x)[EPL])
{
    const char *row = (v ? p.v_cache : p.k_cache) + blk * p.c_blk + off * p.c_slot + h * p.c_head;
    if constexpr (CK == kU3) {
        const float s = __half2float(__ushort_as_half((v ? p.v_qs : p.k_qs)[blk * p.m_blk + off * p.m_slot + h * p.m_head]));
        const float z = float((v ? p.v_qz : p.k_qz)[blk * p.z_blk + off * p.z_slot + h * p.z_head]);
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int bit = 3 * (e0 + e);
            uint32_t w = uint8_t(row[bit >> 3]);
            if ((bit & 7) > 5) w |= uint32_t(uint8_t(row[(bit >> 3) + 1])) << 8;
            x[e] = (float((w >> (bit & 7)) & 7u) - z) * s;
        }
    } else {
        constexpr int es = is_q8(CK) ? 1 : 2;
        const char *piece = row + (e0 * es >> 4) * p.c_chunk + (e0 * es & 15);
        float s = 1.0f;
        if constexpr (is_q8(CK))
            s = p.scale_mode == 0 ? (v ? p.v_scale : p.k_scale)[h]
                                  : (v ? p.v_gs : p.k_gs)[blk * p.gs_blk + off * p.gs_slot + h * p.gs_head];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            if constexpr (CK == kI8)
                x[e] = float(reinterpret_cast<const int8_t *>(piece)[e]) * s;
            else if constexpr (is_q8(CK))
                x[e] = fp8x2_to_float2<CK, 0>(uint32_t(reinterpret_cast<const uint8_t *>(piece)[e])).x * s;
            else
                x[e] = h2f<CK>(reinterpret_cast<const uint16_t *>(piece)[e]);
        }
    }
}

// The elements of `need` (this lane's) of out = softmax(sm_scale q . K^T) V over
// the first `limit` tokens of the sequence whose block-table row is `table`.
// The whole warp calls it; U keys are in flight.
template <int QK, int CK, int D, int U>
__device__ __forceinline__ void prefill_row(const DecodeParams &p, const int32_t *table, int64_t tok, int head, int limit,
                            const bool (&need)[D / 32])
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const int h = head / p.group;
    const uint16_t *qr = reinterpret_cast<const uint16_t *>(p.q + tok * p.q_b + head * p.q_h) + EPL * lane;
    float q[EPL], acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        q[e] = h2f<QK>(qr[e]);
        acc[e] = 0.0f;
    }
    const float ninf = -__int_as_float(0x7f800000);
    float m = ninf, l = 0.0f;
    bool open = true;                               // some needed element is finite yet: what is not stays so
    if (p.num_blocks == 0) limit = 0;
    for (int t0 = 0; t0 < limit && open; t0 += U) {
        float s[U], v[U][EPL], x[U][EPL];
        bool in[U];
        // the keys' loads together: one that is not there loads block 0 and is left out
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = min(t0 + u, limit - 1), off = t & (p.block_size - 1);
            int64_t blk = table[int64_t(t >> p.block_shift) * p.bt_j];
            in[u] = t0 + u < limit && blk >= 0 && blk < p.num_blocks;
            if (!in[u]) blk = 0;
            cached_elems<CK, EPL>(p, false, blk, off, h, EPL * lane, x[u]);
            cached_elems<CK, EPL>(p, true, blk, off, h, EPL * lane, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) s[u] = fmaf(q[e], x[u][e], s[u]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
            s[u] = in[u] ? s[u] * p.scale_log2 : ninf;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s[u] == ninf) continue;
            // a NaN score makes m and every later weight NaN, as the formula does
            const float mn = s[u] > m || isnan(s[u]) ? s[u] : m;
            const float old = m == ninf ? 0.0f : exp2f(m - mn);
            const float w = exp2f(s[u] - mn);
            m = mn;
            l = l * old + w;
#pragma unroll
            for (int e = 0; e < EPL; ++e) acc[e] = fmaf(w, v[u][e], acc[e] * old);
        }
        open = false;
#pragma unroll
        for (int e = 0; e < EPL; ++e) open |= need[e] && isfinite(acc[e]);
        open = __any_sync(0xffffffffu, open);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *o = reinterpret_cast<uint16_t *>(p.out + tok * p.o_b + head * p.o_h) + EPL * lane;
#pragma unroll
    for (int e = 0; e < EPL; ++e)
        if (need[e]) o[e] = f2h<QK>(acc[e] * inv);
}

// A row of `out` that may not be finite.  Its elements that are not are right
// when what made them so lies among the tokens that the row sees.  Where V holds
// such values, in the same column, in the tokens behind the row's limit that its
// tile worked on (limit .. hi), zero weights may have met them: those
// elements are done again from the row's own tokens, until all of them have
// met a value there that is not finite.  So the row's tokens are walked to their
// end only if in some column a token of the few behind them is the first with
// such a value (512 tokens at the end of 262144, 32 q over 8 kv heads of 128, a NaN row
// of V among them: 0.41 s instead of 1.6 ms, e4m3 0.87 s).
template <int QK, int CK, int D, int U>
__device__ __noinline__ void redo_row(const DecodeParams &p, const int32_t *table, int64_t tok, int head, int limit, int hi)
{
    constexpr int EPL = D / 32;
    constexpr uint16_t kInf = QK == kBF16 ? 0x7f80 : 0x7c00;
    const int lane = threadIdx.x & 31;
    const uint16_t *o = reinterpret_cast<const uint16_t *>(p.out + tok * p.o_b + head * p.o_h) + EPL * lane;
    bool need[EPL], any = false;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        need[e] = (o[e] & kInf) == kInf;
        any |= need[e];
    }
    if (!__any_sync(0xffffffffu, any)) return;
    bool again[EPL], open = true, found = false;    // open: a needed element without such a token
#pragma unroll
    for (int e = 0; e < EPL; ++e) again[e] = false;
    for (int t0 = limit; t0 < hi && open; t0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u;
            const int64_t blk = t < hi ? table[int64_t(t >> p.block_shift) * p.bt_j] : -1;
            if (blk < 0 || blk >= p.num_blocks) continue;
            float x[EPL];
            cached_elems<CK, EPL>(p, true, blk, t & (p.block_size - 1), head / p.group, EPL * lane, x);
#pragma unroll
            for (int e = 0; e < EPL; ++e) again[e] |= need[e] && !isfinite(x[e]);
        }
        open = false;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            open |= need[e] && !again[e];
            found |= again[e];
        }
        open = __any_sync(0xffffffffu, open);
    }
    if (__any_sync(0xffffffffu, found)) prefill_row<QK, CK, D, U>(p, table, tok, head, limit, again);
}

}  // namespace
}  // namespace pkv
